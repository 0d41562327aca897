"""The serving operators around the sparse-attention path, as cases that can be timed and compared.

Four operators: dense causal attention over packed prompts (`prefill`), rows of K and V into and out of a
4-bit paged cache (`kv4`), one decode step over that cache (`decode`: the whole context, `step`: the MSA
step with its index scan), and the care of a paged cache's page tables (`pages`).  `run` computes them in
elementary torch operations, or, where `own` is true, through the framework's calls.

The 4-bit format: a head row of d values has 4 groups of d/4.  A group's scale is one byte with 5 exponent
bits (bias 20) and 3 mantissa bits, 2^(e-20) (1 + m/8), 255 = NaN: the smallest one with 7 scale >= max|x|.
A value is (code - 8) * scale with the code in 1..15 (round to nearest even).  Eight channels make a 32-bit
word whose nibble n holds channel 2n for n < 4 and channel 2(n-4)+1 otherwise.
"""
import math

import torch

own = False

DEV = "cuda"
LO, HI = (0, 4, 1, 5), (2, 6, 3, 7)  # channels in the low and the high nibble of a word's four bytes


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of short chat prompts in one batch, ragged, one of them a single token: latency counts
        dict(name="prefill_chat", op="prefill", lens="331,1,97,640,203", H_q=32, H_kv=8, d=128),
        # an ordinary packed batch of mixed prompts (the varlen mix of the benchmark, 32K tokens in all)
        dict(name="prefill_mix", op="prefill", lens="16000,8000,4001,2500,1200,600,300,167", H_q=32, H_kv=8, d=128),
        # one long document at the 128K workload's head layout
        dict(name="prefill_32k", op="prefill", lens="32768", H_q=64, H_kv=8, d=128),
        # one new token of each of 48 sequences, stored in the step that decodes them
        dict(name="kv4_append", op="kv4", lens=",".join(["1"] * 48), pos=5000, H_kv=8, d=128, page=64),
        # the K and V of a whole packed prompt batch going into the cache after its prefill
        dict(name="kv4_prompt", op="kv4", lens="65000,40961,17000,8111", pos=0, H_kv=8, d=128, page=128),
        # one short conversation at a small head layout: latency counts
        dict(name="decode_chat", op="decode", B=1, ctx=1500, vary=0.0, H_q=8, H_kv=2, d=64, page=64),
        # an ordinary batch of conversations of different lengths
        dict(name="decode_batch", op="decode", B=48, ctx=12000, vary=0.9, H_q=32, H_kv=8, d=128, page=64),
        # the 1M-context decode workload, every key attended
        dict(name="decode_1m", op="decode", B=4, ctx=1 << 20, vary=0.0, H_q=64, H_kv=8, d=128, page=128),
        # the MSA step over contexts of some thousand tokens
        dict(name="step_batch", op="step", B=16, ctx=9000, vary=0.7, H_q=32, H_kv=8, d=128, d_I=64, Bk=64, k=8,
             page=64),
        # the MSA step at the 1M-context decode workload
        dict(name="step_1m", op="step", B=4, ctx=1 << 20, vary=0.0, H_q=64, H_kv=8, d=128, d_I=128, Bk=128, k=16,
             page=128),
        # 8 prompts grow by a token, then 7 more samples of each share their pages
        dict(name="pages_fork", op="pages", what="fork", seqs=8, forks=56, ctx=6000, H_kv=8, d=128, d_I=128, page=128,
             n_pages=1024),
        # half of the sequences have ended: their pages go, the rest move together
        dict(name="pages_compact", op="pages", what="compact", seqs=64, forks=0, ctx=4000, H_kv=8, d=128, d_I=128,
             page=128, n_pages=2560),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "kv4", "decode", "decode", "step", "pages"])
    d, H_kv, gs = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8])
    page = 16 * rng.choice([1, 2, 4, 5, 8, 16])
    if op == "prefill":
        total, n = _log(rng, 16, 14000), _log(rng, 1, 24)
        lens = [max(1, _log(rng, 1, 2 * total // n + 1)) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), H_q=gs * H_kv, H_kv=H_kv, d=d)
    if op == "kv4":
        lens = [_log(rng, 1, 20000) for _ in range(rng.randint(1, 6))] if rng.random() < 0.6 else [1] * _log(rng, 1, 200)
        return dict(op=op, lens=",".join(map(str, lens)), pos=rng.choice([0, _log(rng, 1, 3000)]), H_kv=H_kv, d=d,
                    page=page)
    if op == "decode":
        B, ctx = (_log(rng, 1, 128), _log(rng, 1, 8000)) if rng.random() < 0.6 else (rng.randint(1, 3), _log(rng, 8000, 400000))
        return dict(op=op, B=B, ctx=ctx, vary=rng.choice([0.0, 0.5, 0.95]), H_q=gs * H_kv, H_kv=H_kv, d=d, page=page)
    if op == "step":
        B, ctx = (_log(rng, 1, 32), _log(rng, 1, 20000)) if rng.random() < 0.6 else (rng.randint(1, 3), _log(rng, 20000, 400000))
        return dict(op=op, B=B, ctx=ctx, vary=rng.choice([0.0, 0.5, 0.95]), H_q=gs * H_kv, H_kv=H_kv, d=d,
                    d_I=rng.choice([64, 128]), Bk=rng.choice([64, 128]), k=rng.randint(1, 20), page=page)
    seqs, ctx = rng.randint(1, 40), _log(rng, 1, 4000)
    need = seqs * (-(-(ctx + 1) // page))
    what = rng.choice(["fork", "compact"])
    forks = rng.randint(1, 60) if what == "fork" else 0
    return dict(op="pages", what=what, seqs=seqs, forks=forks, ctx=ctx, H_kv=rng.choice([1, 2, 4]), d=d, d_I=64, page=page,
                n_pages=need + forks + rng.randint(1, need + 8))


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _ctx(case):
    """Context lengths: from (1 - vary) ctx to ctx, the first one ctx itself."""
    B, ctx, lo = case["B"], case["ctx"], case["ctx"] * (1.0 - case["vary"])
    return [max(1, int(ctx - (ctx - lo) * ((i * 37) % B) / max(1, B))) for i in range(B)]


# ---------------------------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _paged(gen, ctx, page, spare):
    """A page table of shuffled pages for the given lengths (unused entries -1), and the number of pages."""
    counts = [-(-c // page) for c in ctx]
    n_pages, most = sum(counts) + spare, max(max(counts), 1)
    ids = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(ctx), most), -1, dtype=torch.int32, device=DEV)
    rows = torch.repeat_interleave(torch.arange(len(ctx)), torch.tensor(counts)).to(DEV)
    cols = torch.cat([torch.arange(c) for c in counts]).to(DEV)
    table[rows, cols] = ids[:sum(counts)]
    return table, n_pages


def _kv4_pool(gen, n_pages, page, H_kv, d):
    """Pools as the cache holds them: codes over their whole range, scales about the maxima of normal rows / 7."""
    pool = {}
    for n in ("k", "v"):
        pool[n + "_codes"] = torch.randint(0, 256, (n_pages, page, H_kv, d // 2), generator=gen, device=DEV,
                                           dtype=torch.uint8)
        pool[n + "_scales"] = torch.randint(136, 156, (n_pages, page, H_kv, 4), generator=gen, device=DEV,
                                            dtype=torch.uint8)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case=case, **{n: case[n] for n in ("H_q", "H_kv", "d", "page") if n in case})
    op = case["op"]
    if op == "prefill":
        lens = _lens(case)
        s["cu_host"] = [sum(lens[:i]) for i in range(len(lens) + 1)]
        N = s["cu_host"][-1]
        s["cu"] = torch.tensor(s["cu_host"], dtype=torch.int32, device=DEV)
        s["q"] = _normal(gen, N, case["H_q"], case["d"])
        s["k"], s["v"] = _normal(gen, N, case["H_kv"], case["d"]), _normal(gen, N, case["H_kv"], case["d"])
        s["scale"] = 1.0 / math.sqrt(case["d"])
    elif op == "kv4":
        lens = _lens(case)
        cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
        N, pos = cu[-1], [case["pos"] + (17 * i) % 61 if case["pos"] else 0 for i in range(len(lens))]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
        s["table"], s["n_pages"] = _paged(gen, [p + n for p, n in zip(pos, lens)], case["page"], 8)
        # a few channels of K are much larger than the rest, as in trained models
        s["k"], s["v"] = _normal(gen, N, case["H_kv"], case["d"]), _normal(gen, N, case["H_kv"], case["d"])
        s["k"][:, :, :: case["d"] // 4] *= 8
        s |= {n: torch.zeros_like(t) for n, t in _kv4_pool(gen, s["n_pages"], case["page"], case["H_kv"], case["d"]).items()}
    elif op in ("decode", "step"):
        s["ctx_host"] = _ctx(case)
        s["ctx"] = torch.tensor(s["ctx_host"], dtype=torch.int32, device=DEV)
        s["table"], s["n_pages"] = _paged(gen, s["ctx_host"], case["page"], 8)
        s |= _kv4_pool(gen, s["n_pages"], case["page"], case["H_kv"], case["d"])
        s["q"] = _normal(gen, case["B"], case["H_q"], case["d"])
        s["scale"] = 1.0 / math.sqrt(case["d"])
        if op == "step":
            # index vectors on a grid of 1/16: their products and sums are exact in 32 bits in any order, so that
            # the block sets are one answer; a few keys are far larger, as the keys that a query looks for are
            grid = lambda *sh: (_normal(gen, *sh).float() * 16).round().clamp(-64, 64).div(16).to(torch.bfloat16)  # noqa: E731
            s["k_idx"], s["q_idx"] = grid(s["n_pages"], case["page"], case["d_I"]), grid(case["B"], case["H_kv"], case["d_I"])
            s["k_idx"][::7, 3] *= 2
    else:
        page, n_pages, seqs, forks = case["page"], case["n_pages"], case["seqs"], case["forks"]
        ctx = [max(1, case["ctx"] - (29 * i) % max(1, case["ctx"] // 3)) for i in range(seqs)]
        table, _ = _paged(gen, ctx, page, 0)
        ids = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        most = -(-(case["ctx"] + 1) // page)
        s["table0"] = torch.full((seqs + forks, most), -1, dtype=torch.int32, device=DEV)
        s["table0"][:seqs, :table.shape[1]] = torch.where(table >= 0, ids[table.clamp_min(0).long()], table)
        s["ctx0"] = torch.tensor(ctx + [0] * forks, dtype=torch.int32, device=DEV)
        s["refs0"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
        for n in ("table", "ctx", "refs"):
            s[n] = torch.empty_like(s[n + "0"])
        shapes = dict(k_idx=(case["d_I"],), k=(case["H_kv"], case["d"]), v=(case["H_kv"], case["d"]))
        s["pools"] = {n: _normal(gen, n_pages, page, *sh) for n, sh in shapes.items()}
        s["grow"] = torch.arange(seqs, dtype=torch.int32, device=DEV)
        s["grow_len"] = s["ctx0"][:seqs] + 1
        s["src"] = torch.arange(forks, dtype=torch.int32, device=DEV) % seqs
        s["dst"] = torch.arange(seqs, seqs + forks, dtype=torch.int32, device=DEV)
        s["ended"] = torch.arange(0, seqs, 2, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _softmax_av(x, v):
    """Rows of scores x [..., n] (-inf = not seen) and values v [..., n, d]: (x's softmax) v and log-sum-exp."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l, (m + torch.log(l)).squeeze(-1)


def _plain_prefill(s):
    q, k, v, gs = s["q"], s["k"], s["v"], s["H_q"] // s["H_kv"]
    out = torch.empty_like(q)
    lse = torch.empty((s["H_q"], q.shape[0]), dtype=torch.float32, device=DEV)
    for a, b in zip(s["cu_host"], s["cu_host"][1:]):  # a sequence sees itself only
        at = torch.arange(b - a, device=DEV)
        unseen = at[None, :] > at[:, None]
        for g in range(s["H_kv"]):  # one group's scores at a time: 64 heads of 32K would not fit
            heads = slice(g * gs, (g + 1) * gs)
            x = q[a:b, heads].float().transpose(0, 1) @ k[a:b, g].float().T * s["scale"]
            o, lse[heads, a:b] = _softmax_av(x.masked_fill_(unseen, -math.inf), v[a:b, g].float())
            out[a:b, heads] = o.transpose(0, 1).to(torch.bfloat16)
    return {"out": out, "lse": lse}


def _scale_value(byte):
    v = ((byte.int() << 20) + ((127 - 20) << 23)).view(torch.float32)  # the byte is the top of an fp32 of that value
    return torch.where(byte == 255, torch.full_like(v, math.nan), v)


def _decode_rows(codes, scales):
    """Values (fp32) of rows of codes [..., d/2] and scales [..., 4]."""
    b = codes.unflatten(-1, (-1, 4))
    c = torch.empty(*b.shape[:-1], 8, dtype=torch.float32, device=codes.device)
    c[..., LO] = (b & 15).float()
    c[..., HI] = (b >> 4).float()
    c = c.flatten(-2).unflatten(-1, (4, -1))
    return ((c - 8) * _scale_value(scales)[..., None]).flatten(-2)


def _encode_rows(x):
    """codes [..., d/2] and scales [..., 4] of rows x [..., d]."""
    g = x.float().unflatten(-1, (4, -1))
    amax = g.abs().amax(-1)
    byte = ((amax / 7).view(torch.int32) >> 20) - (107 << 3)  # 3 mantissa bits of max / 7, cut off
    byte = byte.clamp(0, 254).to(torch.uint8)
    byte = (byte + (7 * _scale_value(byte) < amax).to(torch.uint8)).clamp(max=254)
    c = torch.round(g / _scale_value(byte)[..., None]).clamp(-7, 7) + 8
    bad = ~torch.isfinite(amax)
    byte, c = torch.where(bad, 255, byte), torch.where(bad[..., None], 8.0, c)
    c = c.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 8))
    return (c[..., LO] | (c[..., HI] << 4)).flatten(-2), byte.to(torch.uint8)


def _rows_of(s, N):
    """The pool row of each of N packed rows."""
    at = torch.arange(N, device=DEV)
    seq = torch.searchsorted(s["cu"].long(), at, right=True) - 1
    pos = s["pos"].long()[seq] + at - s["cu"].long()[seq]
    return s["table"].long()[seq, pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_kv4(s):
    rows, out = _rows_of(s, s["k"].shape[0]), {}
    for n in ("k", "v"):
        codes, scales = s[n + "_codes"].flatten(0, 1), s[n + "_scales"].flatten(0, 1)
        codes[rows], scales[rows] = _encode_rows(s[n])
        out[n] = _decode_rows(codes[rows], scales[rows]).to(torch.bfloat16)
    return out


def _cache_rows(s, b, at):
    """K and V (fp32, [len(at), H_kv, d]) of the tokens `at` of sequence b."""
    rows = s["table"][b].long()[at // s["page"]] * s["page"] + at % s["page"]
    return [_decode_rows(s[n + "_codes"].flatten(0, 1)[rows], s[n + "_scales"].flatten(0, 1)[rows]) for n in ("k", "v")]


def _plain_decode(s):
    gs, outs = s["H_q"] // s["H_kv"], []
    for b, n in enumerate(s["ctx_host"]):  # one sequence's cache in fp32 at a time
        k, v = _cache_rows(s, b, torch.arange(n, device=DEV))
        q = s["q"][b].float().unflatten(0, (s["H_kv"], gs))
        outs.append(_softmax_av(q @ k.permute(1, 2, 0) * s["scale"], v.transpose(0, 1)))
    return {"out": torch.stack([o.flatten(0, 1) for o, _ in outs]).to(torch.bfloat16),
            "lse": torch.stack([l.flatten() for _, l in outs])}


def _plain_step(s):
    c, gs, G = s["case"], s["H_q"] // s["H_kv"], s["H_kv"]
    Bk, kb, outs = c["Bk"], c["k"], []
    for b, n in enumerate(s["ctx_host"]):
        at, local = torch.arange(n, device=DEV), (n - 1) // Bk
        rows = s["table"][b].long()[at // s["page"]] * s["page"] + at % s["page"]
        x = s["q_idx"][b].float() @ s["k_idx"].flatten(0, 1)[rows[:local * Bk]].float().T
        best = torch.sort(x.unflatten(1, (local, Bk)).amax(2) if local else x, dim=1, descending=True, stable=True).indices
        blocks = torch.full((G, kb), -1, dtype=torch.int32, device=DEV)
        blocks[:, 0] = local
        blocks[:, 1:1 + min(kb - 1, local)] = best[:, :kb - 1].int()
        tok = (blocks[:, :, None] * Bk + torch.arange(Bk, device=DEV)).flatten(1)  # [G, k Bk]
        seen = (blocks >= 0).repeat_interleave(Bk, 1) & (tok < n)
        k, v = _cache_rows(s, b, tok.clamp(0, n - 1).flatten().long())
        own_group = torch.arange(G, device=DEV)[:, None].expand_as(tok).flatten()
        pick = torch.arange(tok.numel(), device=DEV)
        k, v = k[pick, own_group].unflatten(0, (G, -1)), v[pick, own_group].unflatten(0, (G, -1))
        xs = s["q"][b].float().unflatten(0, (G, gs)) @ k.transpose(1, 2) * s["scale"]
        outs.append((*_softmax_av(xs.masked_fill(~seen[:, None], -math.inf), v), blocks))
    return {"out": torch.stack([o[0].flatten(0, 1) for o in outs]).to(torch.bfloat16),
            "lse": torch.stack([o[1].flatten() for o in outs]), "blocks": torch.stack([o[2] for o in outs])}


def _plain_reserve(s, seqs, lens):
    table, ctx, refs, page = s["table"], s["ctx"], s["refs"], s["page"]
    have, want = -(-ctx[seqs] // page), -(-lens // page)
    col = torch.arange(table.shape[1], device=DEV)
    new = (col >= have[:, None]) & (col < want[:, None])
    free = torch.nonzero(refs == 0).flatten()[:int(new.sum())]
    rows = table[seqs]
    rows[new] = free.int()
    table[seqs], refs[free], ctx[seqs] = rows, 1, lens


def _plain_fork(s, src, dst):
    table, ctx, refs, page = s["table"], s["ctx"], s["refs"], s["page"]
    n, part = ctx[src] // page, (ctx[src] % page) > 0
    rows = table[src]
    shared = torch.arange(table.shape[1], device=DEV) < n[:, None]
    refs += torch.bincount(rows[shared].long(), minlength=refs.numel()).int()
    free = torch.nonzero(refs == 0).flatten()[:int(part.sum())]
    new = torch.where(shared, rows, -1)
    last = n[part].long()
    which = torch.nonzero(part).flatten()
    new[which, last] = free.int()
    for p in s["pools"].values():
        p[free] = p[rows[which, last].long()]
    table[dst], refs[free], ctx[dst] = new, 1, ctx[src]


def _plain_free(s, seqs):
    rows = s["table"][seqs]
    s["refs"] -= torch.bincount(rows[rows >= 0].long(), minlength=s["refs"].numel()).int()
    s["table"][seqs], s["ctx"][seqs] = -1, 0


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n_live = int(live.sum())
    holes = torch.nonzero(~live[:n_live]).flatten()
    moved = torch.nonzero(live[n_live:]).flatten() + n_live
    to = torch.where(live, torch.arange(refs.numel(), device=DEV), -1)
    to[moved] = holes
    for p in s["pools"].values():
        p[holes] = p[moved]
    refs[holes], refs[moved] = refs[moved].clone(), 0
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].int(), table))
    return {"page_map": to.int(), "n_live": torch.tensor([n_live], dtype=torch.int32, device=DEV)}


def _plain_pages(s):
    if s["case"]["what"] == "fork":
        _plain_reserve(s, s["grow"].long(), s["grow_len"])
        _plain_fork(s, s["src"].long(), s["dst"].long())
        return {}
    _plain_free(s, s["ended"].long())
    return _plain_compact(s)


# ---------------------------------------------------------------------------------------------- the framework's calls
def _plan(s):
    """What a serving program keeps between steps: the objects that own workspaces and outputs."""
    if "plan" not in s:
        from block_sparse_long_index_gb300 import api
        c = s["case"]
        if c["op"] == "prefill":
            s["plan"] = api.MsaDensePrefill(s["q"].shape[0], s["H_q"], s["H_kv"], s["d"], s["cu"].numel() - 1)
        elif c["op"] == "pages":
            s["plan"] = api.PagedCache(s["table"], s["ctx"], s["refs"], s["page"], list(s["pools"].values()))
        else:
            pool = api.Kv4Pool(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
            s["plan"] = pool if c["op"] == "kv4" else api.MsaDecodeKv4(
                pool, c["B"], s["table"].shape[1], s["H_q"],
                **({} if c["op"] == "decode" else dict(d_I=c["d_I"], Bk=c["Bk"], k=c["k"])))
    return s["plan"]


def _own_prefill(s):
    out, lse = _plan(s)(s["q"], s["k"], s["v"], s["cu"], s["scale"])
    return {"out": out, "lse": lse}


def _own_kv4(s):
    pool = _plan(s)
    pool.store(s["k"], s["v"], s["cu"], s["pos"], s["table"])
    k, v = pool.load(s["k"].shape[0], s["cu"], s["pos"], s["table"])
    return {"k": k, "v": v}


def _own_decode(s):
    out, lse = _plan(s).dense(s["q"], s["table"], s["ctx"], s["scale"])
    return {"out": out, "lse": lse}


def _own_step(s):
    out, lse, blocks = _plan(s)(s["q"], s["q_idx"], s["k_idx"], s["table"], s["ctx"], s["scale"])
    return {"out": out, "lse": lse, "blocks": blocks}


def _own_pages(s):
    cache = _plan(s)
    if s["case"]["what"] == "fork":
        cache.reserve(s["grow"], s["grow_len"])
        cache.fork(s["src"], s["dst"])
        return {}
    cache.free(s["ended"])
    page_map, n_live = cache.compact()
    return {"page_map": page_map, "n_live": n_live}


def run(state):
    op = state["case"]["op"]
    if op == "pages":
        for n in ("table", "ctx", "refs"):  # every pass starts from the same tables
            state[n].copy_(state[n + "0"])
        got = (_own_pages if own else _plain_pages)(state)
        return {**got, **{n: state[n] for n in ("table", "ctx", "refs")}, **state["pools"]}
    plain, mine = {"prefill": (_plain_prefill, _own_prefill), "kv4": (_plain_kv4, _own_kv4),
                   "decode": (_plain_decode, _own_decode), "step": (_plain_step, _own_step)}[op]
    return (mine if own else plain)(state)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case.get("d", 0)
    row = d // 2 + 4  # bytes of a 4-bit head row
    if op == "prefill":
        lens, H_q, H_kv = _lens(case), case["H_q"], case["H_kv"]
        return {"bytes": sum(lens) * (2 * H_q * d * 2 + 2 * H_kv * d * 2 + 4 * H_q),
                "flops": sum(n * (n + 1) // 2 for n in lens) * H_q * 4 * d}
    if op == "kv4":
        rows = sum(_lens(case)) * case["H_kv"] * 2
        return {"bytes": rows * (2 * d + row + row + 2 * d), "flops": rows * 6 * d}
    if op == "decode":
        n = sum(_ctx(case))
        io = case["B"] * case["H_q"] * (4 * d + 4)
        return {"bytes": n * case["H_kv"] * 2 * row + io, "flops": n * case["H_q"] * 4 * d}
    if op == "step":
        ctx, G = _ctx(case), case["H_kv"]
        seen = sum(min(case["k"] * case["Bk"], n) for n in ctx)
        io = case["B"] * (case["H_q"] * (4 * d + 4) + G * (2 * case["d_I"] + 4 * case["k"]))
        return {"bytes": sum(ctx) * 2 * case["d_I"] + seen * G * 2 * row + io,
                "flops": sum(ctx) * G * 2 * case["d_I"] + seen * case["H_q"] * 4 * d}
    page, seqs = case["page"], case["seqs"]
    ctx = [max(1, case["ctx"] - (29 * i) % max(1, case["ctx"] // 3)) for i in range(seqs)]
    page_bytes = page * 2 * (case["d_I"] + 2 * case["H_kv"] * d)
    most = -(-(case["ctx"] + 1) // page)
    tables = 2 * 4 * ((seqs + case["forks"]) * (most + 1) + case["n_pages"])
    if case["what"] == "fork":
        copies = sum((ctx[i % seqs] + 1) % page > 0 for i in range(case["forks"]))
    else:  # live pages are spread evenly: those past the first n_live move
        n_live = sum(-(-n // page) for n in ctx[1::2])
        copies = n_live * (case["n_pages"] - n_live) / case["n_pages"]
    return {"bytes": copies * 2 * page_bytes + tables, "flops": 0}


# ---------------------------------------------------------------------------------------------- 64 bits
def _scales64():
    b = torch.arange(255, device=DEV)
    return torch.pow(2.0, (b // 8 - 20).double()) * (8 + b % 8).double() / 8


def _values64(codes, scales):
    """Rows in 64 bits, channel by channel: channel c of a word sits in nibble c / 2 + 4 (c % 2)."""
    word = codes.to(torch.int64).unflatten(-1, (-1, 4))
    word = word[..., 0] | word[..., 1] << 8 | word[..., 2] << 16 | word[..., 3] << 24
    ch = torch.stack([(word >> 4 * (c // 2 + 4 * (c % 2))) & 15 for c in range(8)], -1).flatten(-2)
    sc = _scales64()[scales.long()]
    return (ch.double() - 8) * sc.repeat_interleave(ch.shape[-1] // 4, -1)


def _attend64(q, k, v, scale, last=None):
    """q [h, n, d], k and v [m, d]; row i sees keys 0 .. last[i] (all of them where last is None)."""
    x = torch.einsum("hnd,md->hnm", q, k) * scale
    if last is not None:
        x = torch.where(torch.arange(k.shape[0], device=DEV) <= last[:, None], x, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("hnm,md->hnd", torch.exp(x - lse[..., None]), v), lse


def exact(case, seed):
    op = case["op"]
    if op == "pages" or (op != "kv4" and work(case)["flops"] > 3e12):
        return None
    s = prepare(case, seed)
    if op == "prefill":
        gs = case["H_q"] // case["H_kv"]
        out, lse = torch.empty_like(s["q"], dtype=torch.float64), torch.empty(case["H_q"], s["q"].shape[0], dtype=torch.float64, device=DEV)
        for a, b in zip(s["cu_host"], s["cu_host"][1:]):
            for h in range(case["H_kv"]):
                for t in range(a, b, 2048):  # rows at a time, each with the keys that it can see
                    e, hs = min(t + 2048, b), slice(h * gs, h * gs + gs)
                    o, l = _attend64(s["q"][t:e, hs].double().transpose(0, 1), s["k"][a:e, h].double(), s["v"][a:e, h].double(),
                                     s["scale"], torch.arange(t - a, e - a, device=DEV))
                    out[t:e, hs], lse[hs, t:e] = o.transpose(0, 1), l
        return {"out": out, "lse": lse}
    if op == "kv4":
        got = {}
        for n in ("k", "v"):
            x = s[n].double().unflatten(-1, (4, -1))
            sc = _scales64()
            i = torch.searchsorted(7 * sc, x.abs().amax(-1).contiguous()).clamp(max=254)
            got[n] = (torch.round(x / sc[i][..., None]).clamp(-7, 7) * sc[i][..., None]).flatten(-2)
        return got
    gs, outs, lses, blocks = case["H_q"] // case["H_kv"], [], [], []
    for b, n in enumerate(s["ctx_host"]):
        pages = s["table"][b, :-(-n // case["page"])].long()
        tok = lambda t: t[pages].flatten(0, 1)[:n]  # noqa: E731
        sets = None
        if op == "step":
            local = (n - 1) // case["Bk"]
            x = torch.einsum("gd,nd->gn", s["q_idx"][b].double(), tok(s["k_idx"])[:local * case["Bk"]].double())
            top = x.reshape(-1, local, case["Bk"]).amax(2).cpu().tolist() if local else [[]] * case["H_kv"]
            sets = [[local] + sorted(range(local), key=lambda j: (-row[j], j))[:case["k"] - 1] for row in top]
            blocks.append([r + [-1] * (case["k"] - len(r)) for r in sets])
        for g in range(case["H_kv"]):
            at = torch.arange(n, device=DEV)
            if sets is not None:
                at = at[torch.isin(at // case["Bk"], torch.tensor(sets[g], device=DEV))]
            k, v = (_values64(tok(s[m + "_codes"])[at, g], tok(s[m + "_scales"])[at, g]) for m in ("k", "v"))
            o, l = _attend64(s["q"][b, g * gs:g * gs + gs].double()[:, None], k, v, s["scale"])
            outs.append(o[:, 0])
            lses.append(l[:, 0])
    got = {"out": torch.stack(outs).reshape(case["B"], case["H_q"], case["d"]), "lse": torch.stack(lses).reshape(case["B"], case["H_q"])}
    if op == "step":
        got["blocks"] = torch.tensor(blocks, dtype=torch.int32, device=DEV)
    return got
