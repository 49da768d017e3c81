"""The measured cases of the serving operators around the token indexer.

Four operators, each reached through the package's binding:

* `plan`      block tables, slot maps and positions of one step, from request lengths
* `rope`      rotary positions of query rows (bf16 or e4m3 with a scale per row), their
              transpose, and of key rows on their way into a paged cache
* `attend`    attention of a ragged batch of new tokens over a paged cache
* `selected`  attention of every query over its own list of tokens

`run` computes them in elementary torch operations (32 bits, 64 for angles), or, where
`own` is true, makes the package's calls.  `exact` computes them from their definitions
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the bookkeeping of one decode step of a serving batch: one token for each sequence
        dict(name="plan_decode", op="plan", n_seq=64, page=64, q_max=1, ctx_max=32768),
        # a packed prefill of many requests, most of them short
        dict(name="plan_prefill", op="plan", n_seq=4096, page=16, q_max=64, ctx_max=2048),
        # index queries of one decode step: 64 heads of 128, the first half of each rotated
        dict(name="rope_decode", op="rope", form="rows", n=64, H=64, d=128, r=64, offset=0,
             interleaved=True, scaled=False),
        # index queries of a prefill chunk for the FP8 scoring call, long-context frequencies
        dict(name="rope_chunk_fp8", op="rope", form="fp8", n=8192, H=64, d=128, r=64, offset=0,
             interleaved=False, scaled=True),
        # the gradient of rotated queries of an odd number of tokens, whole heads of 64
        dict(name="rope_grad", op="rope", form="grad", n=4099, H=32, d=64, r=64, offset=0,
             interleaved=False, scaled=False),
        # keys and values of a chunk into their page pools, the last 64 of 128 elements rotated
        dict(name="append_kv", op="rope", form="kv", n=8192, H=8, d=128, r=64, offset=64,
             interleaved=False, scaled=True, page=64),
        # one token for each of 64 sequences of mixed lengths: the dense decode step
        dict(name="attend_decode", op="attend", n_seq=64, q_max=1, ctx_max=32768, H=64, Hkv=8,
             d=128, page=64, window=0, sinks=0),
        # a prefill chunk at the end of a long prefix, one sequence
        dict(name="attend_chunk", op="attend", n_seq=1, q_max=2048, ctx_max=30720, H=32, Hkv=4,
             d=128, page=64, window=0, sinks=0),
        # a mixed batch of short chunks with heads of 64, a sliding window and visible first tokens
        dict(name="attend_window", op="attend", n_seq=9, q_max=777, ctx_max=3333, H=12, Hkv=4,
             d=64, page=16, window=1000, sinks=4),
        # sparse decode: each new query over its 2048 selected tokens, keys shared by all heads
        dict(name="selected_decode", op="selected", n_seq=64, q_max=1, ctx_max=32768, H=64, Hkv=1,
             d=128, page=64, k=2048),
        # sparse prefill: every query of a chunk over its own 2048 tokens
        dict(name="selected_chunk", op="selected", n_seq=1, q_max=4096, ctx_max=61440, H=64, Hkv=1,
             d=128, page=64, k=2048),
        # short lists of an odd length, heads of 64 in groups, several sequences
        dict(name="selected_groups", op="selected", n_seq=5, q_max=301, ctx_max=2500, H=24, Hkv=4,
             d=64, page=32, k=333),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "attend", "attend", "selected", "selected"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        n_seq = _log(rng, 1, 4096)
        return dict(op=op, n_seq=n_seq, page=page, q_max=_log(rng, 1, max(2, 131072 // n_seq)),
                    ctx_max=_log(rng, 1, 32768))
    if op == "rope":
        form = rng.choice(["rows", "fp8", "grad", "kv", "index"])
        d = rng.choice([32, 64, 128])
        r = rng.choice([x for x in (16, 32, 64, 128) if x <= d])
        offset = rng.choice([0, d - r])
        H = 1 if form == "index" else _log(rng, 1, 64)
        c = dict(op=op, form=form, n=_log(rng, 1, 8192), H=H, d=d, r=r, offset=offset,
                 interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5)
        if form in ("kv", "index"):
            c["page"] = page
        return c
    Hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    if op == "attend":
        n_seq = _log(rng, 1, 64)
        q_max = _log(rng, 1, max(1, 2048 // n_seq))
        ctx = _log(rng, 1, 32768)
        G = rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g * Hkv <= 64])
        while n_seq * (q_max * G * Hkv + 2 * Hkv * d) * (ctx + q_max) > (1 << 31):
            ctx = max(1, ctx // 2)
            q_max = max(1, q_max // 2)
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return dict(op=op, n_seq=n_seq, q_max=q_max, ctx_max=ctx, H=G * Hkv, Hkv=Hkv, d=d,
                    page=page, window=window, sinks=rng.choice([0, 1, 4, 130]) if window else 0)
    n_seq = _log(rng, 1, 64)
    q_max = _log(rng, 1, max(1, 4096 // n_seq))
    k = _log(rng, 1, 4096)
    G = rng.choice([g for g in (1, 2, 5, 8, 16, 64) if g * Hkv <= 128])
    while n_seq * q_max * k * Hkv * (G + d) > (1 << 30):
        q_max, k = max(1, q_max // 2), max(1, k * 2 // 3)
    return dict(op=op, n_seq=n_seq, q_max=q_max, ctx_max=_log(rng, 1, 61440), H=G * Hkv, Hkv=Hkv,
                d=d, page=page, k=k)


# ---------------------------------------------------------------- lengths of a case (host)

def _lens(case):
    """New tokens and earlier tokens of each sequence, from the case alone: ragged
    between a quarter and the whole of the largest, an empty request among many."""
    n, q, c = case["n_seq"], case["q_max"], case["ctx_max"]
    q_lens = [q if i == 0 else 0 if n > 8 and q > 1 and i % 61 == 7 else
              max(1, (q * (1 + (i * 5) % 4) + 3) // 4) for i in range(n)]
    ctx = [c if i == 0 else (c * (1 + (i * 7) % 8)) // 8 - (i * 13) % max(1, c // 8) for i in range(n)]
    return q_lens, [max(0, x) for x in ctx]


def _pages_of(lens, page):
    return [-(-x // page) for x in lens]


def _paged(case, gen):
    """Lengths, block tables (pages in a random order) and the maps of one step."""
    q_lens, ctx = _lens(case)
    page = case["page"]
    seq = [a + b for a, b in zip(q_lens, ctx)]
    nb = _pages_of(seq, page)
    n_pages, width = sum(nb) + 3, max(nb)
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(seq), max(1, width)), dtype=torch.int32, device=DEV)
    nbt = torch.tensor(nb, device=DEV)
    col = torch.arange(table.shape[1], device=DEV)[None]
    mask = col < nbt[:, None]
    table[mask] = perm[:sum(nb)]
    ql = torch.tensor(q_lens, device=DEV)
    cu = torch.zeros(len(seq) + 1, dtype=torch.int32, device=DEV)
    cu[1:] = ql.cumsum(0)
    n_tok = sum(q_lens)
    seq_of = torch.repeat_interleave(torch.arange(len(seq), device=DEV), ql, output_size=n_tok)
    pos = torch.arange(n_tok, device=DEV) - cu[:-1].long()[seq_of] + torch.tensor(ctx, device=DEV)[seq_of]
    return dict(table=table, n_pages=n_pages, cu=cu, n_tok=n_tok,
                lens=torch.tensor(seq, dtype=torch.int32, device=DEV),
                seq_of=seq_of.to(torch.int32), pos=pos.to(torch.int32), max_len=max(seq),
                max_q=max(q_lens))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


# ---------------------------------------------------------------- rotary frequencies

def _inv_freq(r, scaled, base=10000.0, factor=40.0, trained=4096, fast=32.0, slow=1.0):
    """Angle per position of each pair, 64 bits.  `scaled`: pairs that turn fewer than
    `slow` times within the trained length are slowed by `factor`, those above `fast`
    turns are kept, the ones between blended linearly in the pair's index; the
    amplitude grows with the logarithm of the factor."""
    half = r // 2
    f = [base ** (-2.0 * i / r) for i in range(half)]
    if not scaled:
        return f, 1.0
    at = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(at(fast))), min(r - 1, math.ceil(at(slow)))
    out = []
    for i, x in enumerate(f):
        keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(x / factor * (1.0 - keep) + x * keep)
    return out, 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------- prepare

def prepare(case, seed):
    return {"plan": _prep_plan, "rope": _prep_rope, "attend": _prep_attend,
            "selected": _prep_selected}[case["op"]](case, _gen(seed))


def _prep_plan(case, gen):
    """The request lengths, the tables as the earlier steps left them, and the free pages.
    The lengths of this operator are its data, so they are drawn from the seed."""
    n, page, q_max, ctx_max = case["n_seq"], case["page"], case["q_max"], case["ctx_max"]
    q = torch.randint(1, q_max + 1, (n,), generator=gen, device=DEV, dtype=torch.int32)
    if q_max > 1:
        q[torch.rand(n, generator=gen, device=DEV) < 0.02] = 0
    ctx = torch.randint(0, ctx_max + 1, (n,), generator=gen, device=DEV, dtype=torch.int32)
    width = -(-(q_max + ctx_max) // page)
    have = (ctx.long() + page - 1) // page
    n_pages = n * width + 7
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    mask = torch.arange(width, device=DEV)[None] < have[:, None]
    used = (have.cumsum(0) - have)[:, None] + torch.arange(width, device=DEV)[None]
    table[mask] = perm[used[mask]]
    free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    total = have.sum()
    left = n_pages - total
    k = torch.arange(n_pages, device=DEV)
    free = torch.where(k < left, perm[(total + k).clamp(max=n_pages - 1)], free)
    n_tok = n * q_max
    i32 = dict(dtype=torch.int32, device=DEV)
    st = dict(case=case, q=q, ctx=ctx, table=table, free=free, count=left.to(torch.int32).view(1),
              n_tok=n_tok, page=page, count_out=torch.zeros(1, **i32),
              cu=torch.zeros(n + 1, **i32), lens=torch.zeros(n, **i32), granted=torch.zeros(n, **i32),
              pos=torch.zeros(n_tok, **i32), slots=torch.zeros(n_tok, **i32),
              seq_of=torch.zeros(n_tok, **i32))
    return st


def _prep_rope(case, gen):
    n, H, d, r = case["n"], case["H"], case["d"], case["r"]
    f, amp = _inv_freq(r, case["scaled"])
    st = dict(case=case, x=_randn(gen, n, H, d).to(torch.bfloat16), amp=amp,
              inv_freq=torch.tensor(f, dtype=torch.float64, device=DEV),
              pos=(torch.arange(n, device=DEV) + torch.randint(0, 1 << 20, (1,), generator=gen,
                                                               device=DEV)).to(torch.int32))
    if case["form"] in ("kv", "index"):
        page = case["page"]
        n_pages = -(-n // page) + 2
        st["slots"] = torch.randperm(n_pages * page, generator=gen, device=DEV)[:n].to(torch.int32)
        if case["form"] == "kv":
            st["v"] = _randn(gen, n, H, d).to(torch.bfloat16)
            st["k_pages"] = torch.zeros((n_pages, page, H, d), dtype=torch.bfloat16, device=DEV)
            st["v_pages"] = torch.zeros((n_pages, page, H, d), dtype=torch.bfloat16, device=DEV)
        else:
            st["x"] = st["x"].view(n, d)
            st["k_pages"] = torch.zeros((n_pages, page, d), dtype=torch.uint8, device=DEV)
            st["k_scale"] = torch.ones((n_pages, page), dtype=torch.float32, device=DEV)
    return st


def _prep_cache(case, gen):
    st = _paged(case, gen)
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    gain = torch.exp(0.5 * _randn(gen, st["n_tok"], H, 1))
    st["case"] = case
    st["Q"] = (1.5 * gain * _randn(gen, st["n_tok"], H, d)).to(torch.bfloat16)
    st["k_pages"] = _randn(gen, st["n_pages"], page, Hkv, d).to(torch.bfloat16)
    st["v_pages"] = _randn(gen, st["n_pages"], page, Hkv, d).to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(d)
    return st


def _prep_attend(case, gen):
    return _prep_cache(case, gen)


def _prep_selected(case, gen):
    """Lists as the indexer gives them: distinct visible tokens, ascending, -1 behind them.
    Every 1/k of the visible prefix gives one token, which keeps them distinct."""
    st = _prep_cache(case, gen)
    n_tok, k = st["n_tok"], case["k"]
    vis = st["pos"].long()[:, None] + 1
    u = torch.rand((n_tok, k), generator=gen, device=DEV)
    i = torch.arange(k, device=DEV)[None]
    lo, hi = i * vis // k, (i + 1) * vis // k
    tok = torch.minimum(lo + (u * (hi - lo)).long(), hi - 1)
    tok = torch.where(vis >= k, tok, torch.where(i < vis, i, -1))
    st["idx"] = tok.to(torch.int32).contiguous()
    return st


# ---------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _lib():
    from long_context_sparse_block_b200 import _lib as lib
    return lib


def _own_plan(s):
    _lib().misa_plan_step(
        s["q"], s["ctx"], s["table"], s["page"], cu_q=s["cu"], seq_lens=s["lens"],
        positions=s["pos"], slots=s["slots"], seq_of=s["seq_of"], granted=s["granted"],
        free_pages=s["free"], free_count=s["count"], free_count_out=s["count_out"])
    return {n: s[n] for n in ("table", "cu", "lens", "pos", "slots", "seq_of", "granted", "count_out")}


def _own_rope(s):
    c, lib = s["case"], _lib()
    kw = dict(offset=c["offset"], interleaved=c["interleaved"], amplitude=s["amp"])
    if c["form"] in ("rows", "grad"):
        return lib.misa_rope(s["x"], s["pos"], s["inv_freq"], transpose=c["form"] == "grad", **kw)
    if c["form"] == "fp8":
        codes, scale = lib.misa_rope_fp8(s["x"], s["pos"], s["inv_freq"], **kw)
        return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}
    if c["form"] == "kv":
        lib.misa_cache_append(s["x"], s["pos"], s["slots"], s["inv_freq"], s["k_pages"],
                              v=s["v"], v_pages=s["v_pages"], **kw)
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    lib.misa_cache_append(s["x"], s["pos"], s["slots"], s["inv_freq"], s["k_pages"],
                          k_scale=s["k_scale"], **kw)
    return {"k_pages": s["k_pages"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"]}


def _own_attend(s):
    c = s["case"]
    out, lse = _lib().misa_attend_paged(
        s["Q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], scale=s["scale"],
        window=c["window"], sinks=c["sinks"], want_lse=True)
    return {"out": out, "lse": lse}


def _own_selected(s):
    out, lse = _lib().misa_attend_selected(
        s["Q"], s["k_pages"], s["v_pages"], s["table"], s["seq_of"], s["pos"], s["idx"],
        scale=s["scale"], want_lse=True)
    return {"out": out, "lse": lse}


def _plain_plan(s):
    q, ctx, page, n_tok = s["q"].long(), s["ctx"].long(), s["page"], s["n_tok"]
    n = q.numel()
    cu = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    cu[1:] = q.cumsum(0)
    have, want = (ctx + page - 1) // page, (ctx + q + page - 1) // page
    need = want - have
    end = need.cumsum(0)
    count = s["count"].long()
    ok = (need == 0) | (end <= count)
    taken = torch.where(ok, need, 0).sum()
    first = end - need
    width = s["table"].shape[1]
    col = torch.arange(width, device=DEV)[None]
    fresh = (col >= have[:, None]) & (col < want[:, None]) & ok[:, None]
    at = count - 1 - first[:, None] - (col - have[:, None])
    table = torch.where(fresh, s["free"].long()[at.clamp(0, s["free"].numel() - 1)], s["table"].long())
    t = torch.arange(n_tok, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    live = b < n
    bc = b.clamp(max=n - 1)
    live = live & ok[bc]
    pos = ctx[bc] + t - cu[bc]
    slot = table[bc, (pos // page).clamp(max=width - 1)] * page + pos % page
    i32 = lambda x: x.to(torch.int32)
    s["table"].copy_(i32(table))
    return {"table": s["table"], "cu": i32(cu), "lens": i32(torch.where(ok, ctx + q, 0)),
            "pos": i32(torch.where(live, pos, -1)), "slots": i32(torch.where(live, slot, -1)),
            "seq_of": i32(torch.where(live, bc, -1)), "granted": i32(ok),
            "count_out": i32(count - taken)}


def _rotated(s, x):
    """The rotated rows [n, H, d] in 32 bits; angles in 64."""
    c = s["case"]
    r, o = c["r"], c["offset"]
    ang = s["pos"].double()[:, None] * s["inv_freq"][None]
    cos = (s["amp"] * ang.cos()).float()[:, None]
    sin = (s["amp"] * ang.sin()).float()[:, None]
    if c["form"] == "grad":
        sin = -sin
    y = x.float()
    part = y[..., o:o + r]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        rot = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = part[..., :r // 2], part[..., r // 2:]
        rot = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y[..., :o], rot, y[..., o + r:]), -1)


def _codes(y):
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _plain_rope(s):
    c = s["case"]
    x = s["x"] if s["x"].dim() == 3 else s["x"][:, None]
    y = _rotated(s, x)
    if c["form"] in ("rows", "grad"):
        return y.to(torch.bfloat16)
    if c["form"] == "fp8":
        codes, scale = _codes(y)
        return {"codes": codes, "scale": scale}
    at = s["slots"].long()
    if c["form"] == "kv":
        s["k_pages"].view(-1, c["H"], c["d"])[at] = y.to(torch.bfloat16)
        s["v_pages"].view(-1, c["H"], c["d"])[at] = s["v"]
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    codes, scale = _codes(y[:, 0])
    s["k_pages"].view(-1, c["d"])[at] = codes.view(torch.uint8)
    s["k_scale"].view(-1)[at] = scale
    return {"k_pages": s["k_pages"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"]}


def _softmax_parts(sc, vis):
    """Weights and log-sum over the last axis of the visible scores; a row that sees
    nothing has weights of zero and a log-sum of -inf."""
    sc = sc.masked_fill_(~vis, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    return p, z, (z.log() + m).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    H, Hkv, d, page = c["H"], c["Hkv"], c["d"], c["page"]
    G, n_seq, L, nq = H // Hkv, c["n_seq"], s["max_len"], s["max_q"]
    key = torch.arange(L, device=DEV)
    slot = s["table"].long()[:, key // page] * page + key % page                  # [n_seq, L]
    K = s["k_pages"].view(-1, Hkv, d)[slot].permute(0, 2, 3, 1).float()           # [b, j, d, L]
    V = s["v_pages"].view(-1, Hkv, d)[slot].transpose(1, 2).float()               # [b, j, L, d]
    tok = s["cu"].long()[:-1, None] + torch.arange(nq, device=DEV)[None]          # [b, nq]
    live = tok < s["cu"].long()[1:, None]
    tokc = tok.clamp(max=s["n_tok"] - 1)
    Q = s["Q"][tokc].float().view(n_seq, nq, Hkv, G, d).transpose(1, 2)           # [b, j, nq, G, d]
    sc = torch.matmul(Q.reshape(n_seq, Hkv, nq * G, d), K).mul_(s["scale"])
    pos = s["pos"].long()[tokc][:, :, None]
    vis = key[None, None] <= pos
    if c["window"]:
        vis = vis & ((key[None, None] > pos - c["window"]) | (key < c["sinks"])[None, None])
    vis = vis[:, None, :, None].expand(n_seq, 1, nq, G, L).reshape(n_seq, 1, nq * G, L)
    V = V.masked_fill_((key[None] >= s["lens"].long()[:, None])[:, None, :, None], 0.0)
    p, z, lse = _softmax_parts(sc, vis)
    o = torch.matmul(p, V) / torch.where(z == 0, torch.ones_like(z), z)
    o = o.view(n_seq, Hkv, nq, G, d).transpose(1, 2).reshape(n_seq, nq, H, d)
    lse = lse.view(n_seq, Hkv, nq, G).transpose(1, 2).reshape(n_seq, nq, H)
    return {"out": o[live].to(torch.bfloat16), "lse": lse[live]}


def _plain_selected(s):
    c = s["case"]
    H, Hkv, d, page = c["H"], c["Hkv"], c["d"], c["page"]
    G, n = H // Hkv, s["n_tok"]
    idx = s["idx"].long()
    vis = (idx >= 0) & (idx <= s["pos"].long()[:, None])
    at = torch.where(vis, idx, 0)
    slot = s["table"].long()[s["seq_of"].long()[:, None], at // page] * page + at % page
    K = s["k_pages"].view(-1, Hkv, d)[slot].permute(0, 2, 3, 1).float()           # [n, j, d, k]
    V = s["v_pages"].view(-1, Hkv, d)[slot].transpose(1, 2).float()               # [n, j, k, d]
    Q = s["Q"].float().view(n, Hkv, G, d)
    sc = torch.matmul(Q, K).mul_(s["scale"])
    p, z, lse = _softmax_parts(sc, vis[:, None, None])
    o = torch.matmul(p, V) / torch.where(z == 0, torch.ones_like(z), z)
    return {"out": o.view(n, H, d).to(torch.bfloat16), "lse": lse.view(n, H)}


_OWN = {"plan": _own_plan, "rope": _own_rope, "attend": _own_attend, "selected": _own_selected}
_PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "attend": _plain_attend,
          "selected": _plain_selected}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "plan":
        n, tok = case["n_seq"], case["n_seq"] * case["q_max"]
        fresh = n * case["q_max"] // (2 * case["page"])          # pages handed out, about
        return {"bytes": 4.0 * (5 * n + 3 * tok + 2 * fresh), "flops": 0.0}
    if op == "rope":
        n, H, d, r, form = case["n"], case["H"], case["d"], case["r"], case["form"]
        rows = n * H
        by = {"rows": 4.0 * d, "grad": 4.0 * d, "fp8": 3.0 * d + 4, "kv": 8.0 * d,
              "index": 3.0 * d + 4}[form]
        return {"bytes": rows * by + 4.0 * n * (2 if form in ("kv", "index") else 1) + 4.0 * r,
                "flops": rows * 3.0 * r}
    q, ctx = _lens(case)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    io = sum(q) * H * (4.0 * d + 4)
    if op == "attend":
        w, sinks = case["window"], case["sinks"]
        pairs = keys = 0
        for a, c in zip(q, ctx):
            seen = [min(p + 1, w + min(sinks, max(0, p + 1 - w))) if w else p + 1
                    for p in range(c, c + a)]
            pairs += sum(seen)
            first = max(0, c + 1 - w) if w else 0
            keys += 0 if a == 0 else (c + a - first) + min(sinks, first)
        return {"bytes": io + keys * Hkv * 4.0 * d, "flops": 4.0 * d * H * pairs}
    k = case["k"]
    pairs = sum(min(k, p + 1) for a, c in zip(q, ctx) for p in range(c, c + a))
    rows = sum(min(a + c, sum(min(k, p + 1) for p in range(c, c + a))) for a, c in zip(q, ctx))
    return {"bytes": io + 4.0 * sum(q) * k + rows * Hkv * 4.0 * d, "flops": 4.0 * d * H * pairs}


# ---------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "attend": _exact_attend,
            "selected": _exact_selected}[case["op"]](case, st)


def _exact_plan(case, st):
    """Whole numbers have no 64-bit value to be held to beside the plain form's."""
    return None


def _exact_rope(case, st):
    """Every pair as a complex number times A * exp(+-i * angle)."""
    r, o, n = case["r"], case["offset"], case["n"]
    x = st["x"].double().view(n, -1, case["d"])
    sign = -1.0 if case["form"] == "grad" else 1.0
    ang = sign * st["pos"].double()[:, None] * st["inv_freq"][None, :]
    turn = torch.polar(torch.full_like(ang, st["amp"]), ang)[:, None]
    head = x[..., o:o + r].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
    dim = -1 if case["interleaved"] else -2
    z = torch.complex(head.select(dim, 0).contiguous(), head.select(dim, 1).contiguous()) * turn
    y = x.clone()
    y[..., o:o + r] = torch.stack((z.real, z.imag), dim).flatten(-2)
    form = case["form"]
    if form in ("rows", "grad"):
        return y
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    if form == "fp8":
        return {"codes": y / scale[..., None], "scale": scale}
    at = st["slots"].long()
    pages = st["k_pages"].double() if form == "kv" else torch.zeros(
        st["k_pages"].shape, dtype=torch.float64, device=DEV)
    if form == "kv":
        v = st["v_pages"].double()
        pages.view(-1, case["H"], case["d"])[at] = y
        v.view(-1, case["H"], case["d"])[at] = st["v"].double()
        return {"k_pages": pages, "v_pages": v}
    ks = st["k_scale"].double()
    pages.view(-1, case["d"])[at] = (y / scale[..., None])[:, 0]
    ks.view(-1)[at] = scale[:, 0]
    return {"k_pages": pages, "k_scale": ks}


def _exact_rows(q, K, V, vis, scale):
    """One head's rows q [n, d] over K, V [L, d] where vis [n, L]."""
    s = torch.where(vis, (q @ K.T) * scale, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    return w @ V, lse


def _exact_attend(case, st):
    H, Hkv, page = case["H"], case["Hkv"], case["page"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["Q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    q_lens, ctx = _lens(case)
    t0 = 0
    for b, (a, c) in enumerate(zip(q_lens, ctx)):
        n = a + c
        rows = st["table"][b].long()[:, None] * page + torch.arange(page, device=DEV)[None]
        rows = rows.reshape(-1)[:n]
        key = torch.arange(n, device=DEV)[None]
        for i0 in range(0, a, 1024):
            i1 = min(a, i0 + 1024)
            p = (c + torch.arange(i0, i1, device=DEV))[:, None]
            vis = key <= p
            if case["window"]:
                vis &= (key + case["window"] > p) | (key < case["sinks"])
            for j in range(Hkv):
                K = st["k_pages"].view(-1, Hkv, case["d"])[rows, j].double()
                V = st["v_pages"].view(-1, Hkv, case["d"])[rows, j].double()
                for h in range(j * (H // Hkv), (j + 1) * (H // Hkv)):
                    o, l = _exact_rows(st["Q"][t0 + i0:t0 + i1, h].double(), K, V, vis, st["scale"])
                    out[t0 + i0:t0 + i1, h], lse[t0 + i0:t0 + i1, h] = o, l
        t0 += a
    return {"out": out, "lse": lse}


def _exact_selected(case, st):
    H, Hkv, page, d = case["H"], case["Hkv"], case["page"], case["d"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["Q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 22) // case["k"])
    for t0 in range(0, st["n_tok"], step):
        t1 = min(st["n_tok"], t0 + step)
        idx = st["idx"][t0:t1].long()
        keep = (idx >= 0) & (idx <= st["pos"][t0:t1].long()[:, None])
        at = idx.clamp(min=0)
        phys = st["table"][st["seq_of"][t0:t1].long()[:, None].expand_as(at), at // page].long()
        phys = phys * page + at % page
        for j in range(Hkv):
            K = st["k_pages"].view(-1, Hkv, d)[phys, j].double()
            V = st["v_pages"].view(-1, Hkv, d)[phys, j].double()
            hs = slice(j * (H // Hkv), (j + 1) * (H // Hkv))
            s = torch.einsum("ngd,nkd->ngk", st["Q"][t0:t1, hs].double(), K) * st["scale"]
            s = torch.where(keep[:, None], s, -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[..., None])
            out[t0:t1, hs], lse[t0:t1, hs] = torch.einsum("ngk,nkd->ngd", w, V), z
    return {"out": out, "lse": lse}
