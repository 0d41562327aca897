"""The operators of a speculative decode step on paged caches, as cases that can be timed and compared.

Five operators: rotary positions of rows (`rope`), rows of K, V and index keys going into a paged cache with the
rotation applied on the way, beside the step's queries (`append`), attention of a tree of drafted tokens over the cache
(`tree`), the verification of such a tree against the target's probabilities (`verify`), and what then happens to the
cache: the accepted branch stays, the rest goes (`accept`).  `run` computes them in elementary torch operations, or,
where `own` is true, through the framework's calls.

A tree has T nodes a sequence in an order in which parents come first; parents[b, j] < j, -1 for a root.  Node 0 is the
token that the last step ended with, the others are drafts.  Node j of sequence b is token ctx[b] + j of the cache until
it is accepted.

Verification: p[b, n] is the target's distribution after node n, q[b, n] that which the children of n were drawn from.
From node 0 on, the children x of the node n are tested in their order with r = max(0, p - c q), c = 0 and W = 1 at
first: accepted where u q(x) W < r(x); otherwise c grows by W and W becomes the sum of r.  (r / W is what is left of
the target's distribution: each rejection takes max(0, . - q), normalised, of it.)  Without q the drafts were certain:
accepted where u W < r(x), otherwise r(x) becomes 0 and W falls by it.  The walk ends at a node none of whose children
is accepted; the next token is drawn from its r: the lowest one whose cumulative sum exceeds u_last times r's sum.

The 4-bit format: a head row of d values has 4 groups of d/4.  A group's scale is one byte with 5 exponent bits (bias
20) and 3 mantissa bits, 2^(e-20) (1 + m/8), 255 = NaN: the smallest one with 7 scale >= max|x|.  A value is (code - 8)
* scale with the code in 1..15 (round to nearest even).  Eight channels make a 32-bit word whose nibble n holds channel
2n for n < 4 and channel 2(n-4)+1 otherwise.
"""
import math

import torch

own = False

DEV = "cuda"
LO, HI = (0, 4, 1, 5), (2, 6, 3, 7)  # channels in the low and the high nibble of a word's four bytes


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the queries of a decode step of 48 sequences: latency counts
        dict(name="rope_step", op="rope", N=48, H=32, d=128, rot=128, pair="half", dtype="bf16", inverse=False, pos=5000),
        # the gradient of the queries of a 32K training sequence, 64 of whose 128 channels turn, at far positions
        dict(name="rope_grad", op="rope", N=32768, H=64, d=128, rot=64, pair="half", dtype="fp32", inverse=True, pos=900000),
        # a decode step of 48 sequences: queries and index queries turned, a row of K, V and index keys each stored
        dict(name="append_step", op="append", cache="bf16", lens=",".join(["1"] * 48), pos=5000, H_q=32, H_kv=8, d=128,
             rot=128, pair="half", d_I=128, idx="bf16", page=64),
        # the K and V of a packed prompt batch going into the 4-bit cache, its index keys into E4M3
        dict(name="append_prompt", op="append", cache="kv4", lens="65000,40961,17000,8111", pos=0, H_q=0, H_kv=8, d=128,
             rot=64, pair="half", d_I=128, idx="fp8", page=128),
        # one short conversation, eight drafted tokens in a row, at a small head layout: latency counts
        dict(name="tree_chat", op="tree", cache="bf16", B=1, T=8, chain=True, ctx=1500, vary=0.0, H_q=8, H_kv=2, d=64,
             page=64),
        # large trees over conversations of different lengths, bf16 pages
        dict(name="tree_batch", op="tree", cache="bf16", B=16, T=64, chain=False, ctx=12000, vary=0.9, H_q=32, H_kv=8,
             d=128, page=64),
        # small trees over longer conversations in the 4-bit cache
        dict(name="tree_small", op="tree", cache="kv4", B=16, T=8, chain=False, ctx=30000, vary=0.5, H_q=32, H_kv=8,
             d=128, page=64),
        # the 1M-context decode workload with 16 drafted tokens
        dict(name="tree_1m", op="tree", cache="kv4", B=4, T=16, chain=False, ctx=1 << 20, vary=0.0, H_q=64, H_kv=8,
             d=128, page=128),
        # five drafted tokens in a row of one conversation: latency counts
        dict(name="verify_chat", op="verify", B=1, T=6, chain=True, V=50001, drawn=True),
        # trees of a large batch over a large vocabulary
        dict(name="verify_batch", op="verify", B=64, T=24, chain=False, V=128000, drawn=True),
        # a few conversations keep what was accepted of small trees
        dict(name="accept_step", op="accept", B=8, T=8, ctx=3000, H_kv=8, d=128, d_I=128, page=64, layers=1),
        # a large batch with large trees, four layers' pools
        dict(name="accept_batch", op="accept", B=256, T=64, ctx=1200, H_kv=8, d=128, d_I=0, page=64, layers=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "tree", "tree", "tree", "verify", "accept"])
    d, H_kv, gs = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 8])
    page = 16 * rng.choice([1, 2, 4, 5, 8, 16])
    rot, pair = rng.choice([16, 32, 64, 128]), rng.choice(["half", "interleaved"])
    if op == "rope":
        return dict(op=op, N=_log(rng, 1, 30000), H=rng.choice([1, 5, 8, 32]), d=d, rot=min(rot, d), pair=pair,
                    dtype=rng.choice(["bf16", "fp32"]), inverse=rng.random() < 0.5, pos=_log(rng, 1, 2000000))
    if op == "append":
        lens = [_log(rng, 1, 20000) for _ in range(rng.randint(1, 6))] if rng.random() < 0.5 else [rng.randint(1, 64)] * _log(rng, 1, 100)
        return dict(op=op, cache=rng.choice(["bf16", "kv4"]), lens=",".join(map(str, lens)), pos=rng.choice([0, _log(rng, 1, 3000)]),
                    H_q=rng.choice([0, gs * H_kv]), H_kv=H_kv, d=d, rot=min(rot, 64), pair=pair, d_I=rng.choice([0, 64, 128]),
                    idx=rng.choice(["bf16", "fp8"]), page=page)
    if op == "tree":
        B, ctx = (_log(rng, 1, 64), _log(rng, 1, 6000)) if rng.random() < 0.6 else (rng.randint(1, 3), _log(rng, 6000, 200000))
        return dict(op=op, cache=rng.choice(["bf16", "kv4"]), B=B, T=_log(rng, 1, 64), chain=rng.random() < 0.3, ctx=ctx,
                    vary=rng.choice([0.0, 0.5, 0.95]), H_q=gs * H_kv, H_kv=H_kv, d=d, page=page)
    if op == "verify":
        return dict(op=op, B=_log(rng, 1, 48), T=_log(rng, 1, 32), chain=rng.random() < 0.4, V=_log(rng, 100, 160000),
                    drawn=rng.random() < 0.7)
    return dict(op=op, B=_log(rng, 1, 128), T=_log(rng, 1, 64), ctx=_log(rng, 1, 3000), H_kv=H_kv, d=d,
                d_I=rng.choice([0, 64]), page=page, layers=rng.randint(1, 2))


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _ctx(case):
    """Context lengths: from (1 - vary) ctx to ctx, the first one ctx itself."""
    B, ctx, lo = case["B"], case["ctx"], case["ctx"] * (1.0 - case.get("vary", 0.3))
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
        pool[n + "_codes"] = torch.randint(0, 256, (n_pages, page, H_kv, d // 2), generator=gen, device=DEV, dtype=torch.uint8)
        pool[n + "_scales"] = torch.randint(136, 156, (n_pages, page, H_kv, 4), generator=gen, device=DEV, dtype=torch.uint8)
    return pool


def _tree(gen, B, T, chain):
    """Parents [B, T]: a chain, or each draft below one of the few nodes before it."""
    at = torch.arange(T, device=DEV)
    back = torch.ones((B, T), device=DEV) if chain else torch.rand((B, T), generator=gen, device=DEV) * 6 + 1
    return (at - back.long()).clamp_min(0).where(at > 0, -1).to(torch.int32)


def _freqs(rot):
    """Radians a position of each pair, base 10000 in 64 bits."""
    return torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case=case, **{n: case[n] for n in ("H_q", "H_kv", "d", "page", "rot", "T", "B") if n in case})
    op = case["op"]
    if op == "rope":
        x = torch.randn((case["N"], case["H"], case["d"]), generator=gen, device=DEV)
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["positions"] = (torch.arange(case["N"], device=DEV) + case["pos"]).to(torch.int32)
        s["freqs"] = _freqs(case["rot"])
    elif op == "append":
        lens, H_kv, d, d_I = _lens(case), case["H_kv"], case["d"], case["d_I"]
        cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
        N, pos = cu[-1], [case["pos"] + (17 * i) % 61 if case["pos"] else 0 for i in range(len(lens))]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
        s["table"], s["n_pages"] = _paged(gen, [p + n for p, n in zip(pos, lens)], case["page"], 8)
        s["k"], s["v"] = _normal(gen, N, H_kv, d), _normal(gen, N, H_kv, d)
        if case["H_q"]:
            s["q"] = _normal(gen, N, case["H_q"], d)
        if case["cache"] == "bf16":
            s |= {n: torch.zeros((s["n_pages"], case["page"], H_kv, d), dtype=torch.bfloat16, device=DEV) for n in ("k_pool", "v_pool")}
        else:
            s |= {n: torch.zeros_like(t) for n, t in _kv4_pool(gen, s["n_pages"], case["page"], H_kv, d).items()}
        if d_I:
            s["k_idx"] = _normal(gen, N, d_I)
            if case["H_q"]:
                s["q_idx"] = _normal(gen, N, H_kv, d_I)
            idx = torch.bfloat16 if case["idx"] == "bf16" else torch.uint8
            s["k_idx_pool"] = torch.zeros((s["n_pages"], case["page"], d_I), dtype=idx, device=DEV)
        s["freqs"] = _freqs(case["rot"])
    elif op == "tree":
        s["ctx_host"] = _ctx(case)
        s["ctx"] = torch.tensor(s["ctx_host"], dtype=torch.int32, device=DEV)
        s["table"], s["n_pages"] = _paged(gen, [n + case["T"] for n in s["ctx_host"]], case["page"], 8)
        if case["cache"] == "kv4":
            s |= _kv4_pool(gen, s["n_pages"], case["page"], case["H_kv"], case["d"])
        else:
            s |= {n: _normal(gen, s["n_pages"], case["page"], case["H_kv"], case["d"]) for n in ("k_pool", "v_pool")}
        s["q"] = _normal(gen, case["B"], case["T"], case["H_q"], case["d"])
        s["parents"] = _tree(gen, case["B"], case["T"], case["chain"])
        s["scale"] = 1.0 / math.sqrt(case["d"])
    elif op == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        # logits as spread out as a model's, the drafting model's near the target's
        x = torch.randn((B, T, V), generator=gen, device=DEV) * 3
        s["p"] = torch.softmax(x, -1)
        x += torch.randn((B, T, V), generator=gen, device=DEV) * 0.7
        q = torch.softmax(x, -1)
        del x
        s["parents"] = _tree(gen, B, T, case["chain"])
        cum = q.cumsum(-1, dtype=torch.float32)
        up = s["parents"].clamp_min(0).long()
        hit = torch.rand((B, T, 1), generator=gen, device=DEV) * cum[..., -1:].gather(1, up[..., None])
        s["tokens"] = torch.stack([torch.searchsorted(cum[b, up[b]], hit[b]).clamp_max(V - 1)[:, 0] for b in range(B)]).to(torch.int32)
        del cum
        if case["drawn"]:
            s["q"] = q
        s["u"] = torch.rand((B, T), generator=gen, device=DEV)
        s["u_last"] = torch.rand((B,), generator=gen, device=DEV)
    else:
        B, T, page = case["B"], case["T"], case["page"]
        ctx = _ctx(case)
        s["base"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["table0"], n_pages = _paged(gen, [n + T for n in ctx], page, 8)
        s["ctx0"] = s["base"] + T
        s["refs0"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
        for n in ("table", "ctx", "refs"):
            s[n] = torch.empty_like(s[n + "0"])
        shapes = {"k": (case["H_kv"], case["d"]), "v": (case["H_kv"], case["d"])} | ({"k_idx": (case["d_I"],)} if case["d_I"] else {})
        s["pools"] = {"%s%d" % (n, l): _normal(gen, n_pages, page, *sh) for l in range(case["layers"]) for n, sh in shapes.items()}
        # branches as a verification leaves them: some of the nodes, in order, node 0 first
        keep = torch.rand((B, T), generator=gen, device=DEV) < 0.4
        keep[:, 0] = True
        s["n_path"] = keep.sum(1).to(torch.int32)
        at = torch.arange(T, device=DEV)
        s["path"] = torch.where(keep, at, T + at).sort(1).values.where(at < s["n_path"][:, None], -1).to(torch.int32)
        s["seqs"] = torch.arange(B, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _turn(x, positions, freqs, pair, inverse=False):
    """Rows x [N, H, d] with the first 2 len(freqs) channels turned, in fp32; angles in 64 bits."""
    n = freqs.numel()
    angle = positions.double()[:, None] * freqs
    c, sn = torch.cos(angle).float()[:, None], torch.sin(-angle if inverse else angle).float()[:, None]
    x = x.float()
    y = x.clone()
    first, second = (slice(0, n), slice(n, 2 * n)) if pair == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * sn
    y[..., second] = b * c + a * sn
    return y


def _plain_rope(s):
    c = s["case"]
    return {"y": _turn(s["x"], s["positions"], s["freqs"], c["pair"], c["inverse"]).to(s["x"].dtype)}


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
    c = c.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 8))
    return (c[..., LO] | (c[..., HI] << 4)).flatten(-2), byte


def _row_places(s, N):
    """The token position and the pool row of each of N packed rows."""
    at = torch.arange(N, device=DEV)
    seq = torch.searchsorted(s["cu"].long(), at, right=True) - 1
    pos = s["pos"].long()[seq] + at - s["cu"].long()[seq]
    return pos, s["table"].long()[seq, pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_append(s):
    pos, rows = _row_places(s, s["k"].shape[0])
    turned = lambda x: _turn(x, pos, s["freqs"], s["case"]["pair"]).to(torch.bfloat16)  # noqa: E731
    k, out = turned(s["k"]), {}
    if s["case"]["cache"] == "bf16":
        s["k_pool"].flatten(0, 1)[rows], s["v_pool"].flatten(0, 1)[rows] = k, s["v"]
        out |= {n: s[n] for n in ("k_pool", "v_pool")}
    else:
        for n, x in (("k", k), ("v", s["v"])):
            codes, scales = s[n + "_codes"].flatten(0, 1), s[n + "_scales"].flatten(0, 1)
            codes[rows], scales[rows] = _encode_rows(x)
            out[n] = _decode_rows(codes[rows], scales[rows]).to(torch.bfloat16)
    if "q" in s:
        out["q"] = turned(s["q"])
    if "k_idx" in s:
        f8 = s["case"]["idx"] == "fp8"
        held = lambda x: x.float().clamp(-448, 448).to(torch.float8_e4m3fn) if f8 else x  # noqa: E731
        pool = s["k_idx_pool"].view(torch.float8_e4m3fn) if f8 else s["k_idx_pool"]
        idx = held(turned(s["k_idx"][:, None])[:, 0])
        s["k_idx_pool"].flatten(0, 1)[rows] = idx.view(torch.uint8) if f8 else idx
        out["k_idx_pool"] = pool
        if "q_idx" in s:
            out["q_idx"] = held(turned(s["q_idx"]))
    return out


def _tree_mask(parents):
    """seen [B, T, T]: node i sees node j where j is i or above it."""
    B, T = parents.shape
    seen = torch.eye(T, device=DEV).expand(B, T, T)
    up = torch.zeros((B, T, T + 1), device=DEV).scatter(2, parents.long().where(parents >= 0, T)[..., None], 1.0)[..., :T] + seen
    for _ in range(max(1, (T - 1).bit_length())):  # paths of length 1, 2, 4, ...
        up = (up @ up).clamp_max(1)
    return up > 0


def _cache_rows(s, b, at):
    """K and V (fp32, [len(at), H_kv, d]) of the tokens `at` of sequence b."""
    rows = s["table"][b].long()[at // s["page"]] * s["page"] + at % s["page"]
    if "k_pool" in s:
        return [s[n].flatten(0, 1)[rows].float() for n in ("k_pool", "v_pool")]
    return [_decode_rows(s[n + "_codes"].flatten(0, 1)[rows], s[n + "_scales"].flatten(0, 1)[rows]) for n in ("k", "v")]


def _plain_tree(s):
    gs, T, outs, seen = s["H_q"] // s["H_kv"], s["T"], [], _tree_mask(s["parents"])
    for b, n in enumerate(s["ctx_host"]):  # one sequence's cache in fp32 at a time
        k, v = _cache_rows(s, b, torch.arange(n + T, device=DEV))
        q = s["q"][b].float().unflatten(1, (s["H_kv"], gs)).permute(1, 0, 2, 3).flatten(1, 2)  # [H_kv, T gs, d]
        x = q @ k.permute(1, 2, 0) * s["scale"]
        x[..., n:].masked_fill_(~seen[b].repeat_interleave(gs, 0), -math.inf)
        m = x.amax(-1, keepdim=True)
        x = torch.exp(x - m)
        l = x.sum(-1, keepdim=True)
        o = (x @ v.transpose(0, 1)) / l
        outs.append([t.unflatten(1, (T, gs)).transpose(0, 1).flatten(1, 2) for t in (o, m + torch.log(l))])
    return {"out": torch.stack([o for o, _ in outs]).to(torch.bfloat16), "lse": torch.stack([l[..., 0] for _, l in outs])}


def _plain_verify(s):
    p, q, parents, tokens = s["p"], s.get("q"), s["parents"].long(), s["tokens"].long()
    B, T, V = p.shape
    each = torch.arange(B, device=DEV)
    node, c, W = torch.zeros(B, dtype=torch.long, device=DEV), torch.zeros(B, 1, dtype=torch.float64, device=DEV), torch.ones(B, dtype=torch.float64, device=DEV)
    taken = torch.zeros((B, T), dtype=torch.bool, device=DEV)
    taken[:, 0] = True
    row = p[:, 0].double()
    off = torch.zeros((B, V), dtype=torch.bool, device=DEV)  # certain drafts that were rejected
    for j in range(1, T):  # parents come first, so one pass in the nodes' order is the walk
        asked, x = parents[:, j] == node, tokens[:, j]
        left = (row - c * q[each, node].double()).clamp_min(0) if q is not None else row.masked_fill(off, 0)
        r = left[each, x]
        mine = (q[each, node, x].double() if q is not None else 1.0) * s["u"][:, j].double() * W < r
        yes, no = asked & mine, asked & ~mine
        taken[:, j] = yes
        node = torch.where(yes, j, node)
        if q is not None:
            c = torch.where(yes[:, None], 0.0, c + W[:, None] * no[:, None])
            rest = (p[each, node].double() - c * q[each, node].double()).clamp_min(0).sum(1)
        else:
            off[each, x] |= no
            off &= ~yes[:, None]
            rest = W - r
        W = torch.where(yes, 1.0, torch.where(no, rest, W))
        row = p[each, node].double()
    left = (row - c * q[each, node].double()).clamp_min(0) if q is not None else row.masked_fill(off, 0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, row)
    cum = left.cumsum(1)
    nxt = torch.searchsorted(cum, s["u_last"].double()[:, None] * cum[:, -1:], right=True).clamp_max(V - 1)[:, 0]
    at = torch.arange(T, device=DEV)
    n = taken.sum(1)
    path = torch.where(taken, at, T + at).sort(1).values.where(at < n[:, None], -1)
    return {"path": path.int(), "n_path": n.int(), "next": nxt.int()}


def _plain_accept(s):
    page, T, table, ctx = s["page"], s["T"], s["table"], s["ctx"]
    at = torch.arange(T, device=DEV)
    kept = at < s["n_path"][:, None]
    row = lambda t: table.long().gather(1, t // page) * page + t % page  # noqa: E731
    base = s["base"].long()[:, None]
    to, frm = row(base + at)[kept], row(base + s["path"].long().where(kept, at))[kept]
    for p in s["pools"].values():
        p = p.flatten(0, 1)
        p[to] = p[frm]
    new = s["base"] + s["n_path"]
    gone = torch.arange(table.shape[1], device=DEV) >= (-(-new // page))[:, None]
    s["refs"][table[gone & (table >= 0)].long()] = 0
    table.masked_fill_(gone, -1)
    ctx.copy_(new)
    return {}


# ---------------------------------------------------------------------------------------------- the framework's calls
def _plan(s):
    """What a serving program keeps between steps: the objects that own tables, workspaces and outputs."""
    if "plan" not in s:
        from block_sparse_long_index_gb300 import api
        c = s["case"]
        if c["op"] in ("rope", "append"):
            s["rope"] = api.Rope.from_frequencies(s["freqs"], interleaved=c["pair"] == "interleaved")
        if c["op"] in ("append", "tree"):
            s["pool"] = api.KvPool(s["k_pool"], s["v_pool"]) if c["cache"] == "bf16" else api.Kv4Pool(
                s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        s["plan"] = {"rope": lambda: s["rope"], "append": lambda: s["pool"],
                     "tree": lambda: api.MsaTreeDecode(s["pool"], c["B"], c["T"], s["table"].shape[1], c["H_q"]),
                     "verify": lambda: api.DraftVerifier(c["B"], c["T"], c["V"]),
                     "accept": lambda: api.PagedCache(s["table"], s["ctx"], s["refs"], s["page"], list(s["pools"].values()))}[c["op"]]()
    return s["plan"]


def _own_rope(s):
    return {"y": _plan(s)(s["x"], s["positions"], inverse=s["case"]["inverse"])}


def _own_append(s):
    pool, f8 = _plan(s), s["case"]["idx"] == "fp8"
    q, q_idx = pool.append(s["k"], s["v"], s["cu"], s["pos"], s["table"], rope=s["rope"], q=s.get("q"), k_idx=s.get("k_idx"),
                           k_idx_pool=s.get("k_idx_pool"), q_idx=s.get("q_idx"))
    if s["case"]["cache"] == "bf16":
        out = {n: s[n] for n in ("k_pool", "v_pool")}
    else:
        out = dict(zip(("k", "v"), pool.load(s["k"].shape[0], s["cu"], s["pos"], s["table"])))
    if q is not None:
        out["q"] = q
    if "k_idx" in s:
        out["k_idx_pool"] = s["k_idx_pool"].view(torch.float8_e4m3fn) if f8 else s["k_idx_pool"]
    if q_idx is not None:
        out["q_idx"] = q_idx.view(torch.float8_e4m3fn) if f8 else q_idx
    return out


def _own_tree(s):
    out, lse = _plan(s)(s["q"], s["table"], s["ctx"], s["parents"], scale=s["scale"])
    return {"out": out, "lse": lse}


def _own_verify(s):
    path, n_path, nxt = _plan(s)(s["p"], s["tokens"], s["parents"], s["u"], s["u_last"], draft_probs=s.get("q"))
    return {"path": path, "n_path": n_path, "next": nxt}


def _own_accept(s):
    _plan(s).accept(s["seqs"], s["base"], s["path"], s["n_path"])
    return {}


def run(state):
    op = state["case"]["op"]
    if op == "accept":
        for n in ("table", "ctx", "refs"):  # every pass starts from the same tables
            state[n].copy_(state[n + "0"])
        (_own_accept if own else _plain_accept)(state)
        return {**{n: state[n] for n in ("table", "ctx", "refs")}, **state["pools"]}
    plain, mine = {"rope": (_plain_rope, _own_rope), "append": (_plain_append, _own_append), "tree": (_plain_tree, _own_tree),
                   "verify": (_plain_verify, _own_verify)}[op]
    return (mine if own else plain)(state)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case.get("d", 0)
    if op == "rope":
        n = case["N"] * case["H"] * d * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": 2 * n + 4 * case["N"], "flops": case["N"] * case["H"] * case["rot"] * 3}
    row = 2 * d if case.get("cache") == "bf16" else d // 2 + 4  # bytes of a cached head row
    if op == "append":
        N, H_kv, d_I = sum(_lens(case)), case["H_kv"], case["d_I"]
        held = 2 if case["idx"] == "bf16" else 1
        # K and V in and out (a 4-bit cache's rows are read back too, as values), queries, index rows
        each = 2 * H_kv * (2 * d + row + (row + 2 * d if case["cache"] == "kv4" else 0)) + case["H_q"] * 4 * d
        each += d_I * (2 + held) * (1 + (H_kv if case["H_q"] else 0))
        return {"bytes": N * each, "flops": N * (H_kv + case["H_q"]) * case["rot"] * 3}
    if op == "tree":
        n, T = sum(_ctx(case)), case["T"]
        io = case["B"] * T * (case["H_q"] * (4 * d + 4) + 2 * case["H_kv"] * row + 4)
        return {"bytes": n * case["H_kv"] * 2 * row + io, "flops": n * T * case["H_q"] * 4 * d}
    if op == "verify":  # the distributions of the node that the walk ends at
        return {"bytes": case["B"] * (case["V"] * (8 if case["drawn"] else 4) + 16 * case["T"]), "flops": case["B"] * case["V"] * 3}
    token = 2 * (2 * case["H_kv"] * d + case["d_I"]) * case["layers"]
    moved = case["B"] * 0.4 * (case["T"] - 1)
    return {"bytes": 2 * moved * token + 8 * case["B"] * case["T"] + 4 * case["B"], "flops": 0}


# ---------------------------------------------------------------------------------------------- 64 bits
def _turned64(x, pos, freqs, pair, sign=1.0):
    """Rows as complex numbers, one a pair, multiplied by e^(i angle)."""
    x, n = x.double(), freqs.numel()
    turn, rest = x[..., :2 * n], x[..., 2 * n:]
    z = turn.unflatten(-1, (2, n)).transpose(-1, -2) if pair == "half" else turn.unflatten(-1, (n, 2))
    z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones((), dtype=torch.float64, device=DEV), sign * pos.double()[:, None, None] * freqs)
    z = torch.view_as_real(z)
    z = z.transpose(-1, -2).flatten(-2) if pair == "half" else z.flatten(-2)
    return torch.cat([z, rest], -1)


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


def _four_bits64(x):
    x = x.double().unflatten(-1, (4, -1))
    sc = _scales64()
    i = torch.searchsorted(7 * sc, x.abs().amax(-1).contiguous()).clamp(max=254)
    return (torch.round(x / sc[i][..., None]).clamp(-7, 7) * sc[i][..., None]).flatten(-2)


def _exact_append(case, s):
    lens, pos = _lens(case), s["pos"].tolist()
    at = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(pos, lens)])
    rows = torch.cat([(s["table"][i].long()[:, None] * case["page"] + torch.arange(case["page"], device=DEV)).flatten()[p:p + n]
                      for i, (p, n) in enumerate(zip(pos, lens))])
    turned = lambda x: _turned64(x, at, s["freqs"], case["pair"])  # noqa: E731
    bf16 = lambda x: x.to(torch.bfloat16).double()  # noqa: E731  what is stored is what the rotated rows are as bf16
    into = lambda x, n: torch.zeros((n, *x.shape[1:]), dtype=torch.float64, device=DEV).index_put_((rows,), x)  # noqa: E731
    slots, got = s["n_pages"] * case["page"], {}
    if case["cache"] == "bf16":
        got["k_pool"] = into(turned(s["k"]), slots).unflatten(0, (-1, case["page"]))
        got["v_pool"] = into(s["v"].double(), slots).unflatten(0, (-1, case["page"]))
    else:
        got["k"], got["v"] = _four_bits64(bf16(turned(s["k"]))), _four_bits64(s["v"])
    if "q" in s:
        got["q"] = turned(s["q"])
    if "k_idx" in s:
        got["k_idx_pool"] = into(turned(s["k_idx"][:, None])[:, 0], slots).unflatten(0, (-1, case["page"]))
        if "q_idx" in s:
            got["q_idx"] = turned(s["q_idx"])
    return got


def exact(case, seed):
    op = case["op"]
    if op in ("verify", "accept") or work(case)["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    if op == "rope":
        return {"y": _turned64(s["x"], s["positions"], s["freqs"], case["pair"], -1.0 if case["inverse"] else 1.0)}
    if op == "append":
        return _exact_append(case, s)
    gs, T, parents = case["H_q"] // case["H_kv"], case["T"], s["parents"].tolist()
    out = torch.empty((case["B"], T, case["H_q"], case["d"]), dtype=torch.float64, device=DEV)
    lse = torch.empty((case["B"], T, case["H_q"]), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["ctx_host"]):
        pages = s["table"][b, :-(-(n + T) // case["page"])].long()
        tok = lambda t: t[pages].flatten(0, 1)[:n + T]  # noqa: E731
        sees = torch.zeros((T, n + T), dtype=torch.bool)
        sees[:, :n] = True
        for i in range(T):
            j = i
            while j >= 0:
                sees[i, n + j] = True
                j = parents[b][j]
        sees = sees.to(DEV)
        for g in range(case["H_kv"]):
            k, v = ((tok(s[m + "_pool"])[:, g].double() if case["cache"] == "bf16" else
                     _values64(tok(s[m + "_codes"])[:, g], tok(s[m + "_scales"])[:, g])) for m in ("k", "v"))
            for h in range(g * gs, g * gs + gs):
                x = (s["q"][b, :, h].double() @ k.T * s["scale"]).masked_fill(~sees, -math.inf)
                lse[b, :, h] = torch.logsumexp(x, -1)
                out[b, :, h] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}
