"""Verification of drafted trees and the accepted branch on the GPU, and the steps of speculative decoding run together."""
import math

import numpy as np
import pytest
import torch

import draft_ref as ref
from test_gpu_kv4 import i32
from test_gpu_rope import rows

pytestmark = pytest.mark.gpu


def trees(rng, B, T, V, kind, drawn, spread=3.0):
    """probs, draft_probs (fp32, numpy), tokens, parents, u, u_last of B sequences, the drafts drawn from draft_probs."""
    x = rng.standard_normal((B, T, V)) * spread
    soft = lambda z: (lambda e: (e / e.sum(-1, keepdims=True)).astype(np.float32))(np.exp(z - z.max(-1, keepdims=True)))  # noqa: E731
    p, q = soft(x), soft(x + rng.standard_normal((B, T, V)) * 0.7)
    parents = np.array([ref.tree_of(rng, T, kind) for _ in range(B)], np.int32)
    tokens = np.zeros((B, T), np.int32)
    for b in range(B):
        for j in range(1, T):
            w = q[b, max(parents[b, j], 0)].astype(np.float64)
            tokens[b, j] = rng.choice(V, p=w / w.sum())
    u, ul = rng.random((B, T)).astype(np.float32), rng.random(B).astype(np.float32)
    return p, (q if drawn else None), tokens, parents, np.minimum(u, np.float32(0.9999999)), np.minimum(ul, np.float32(0.9999999))


def call(p, q, tokens, parents, u, ul, tree_len=None, run=None):
    from block_sparse_long_index_gb300 import DraftVerifier
    dev = lambda a: None if a is None else torch.tensor(a, device="cuda")  # noqa: E731
    B, T, V = p.shape
    run = run or DraftVerifier(B, T, V)
    path, n, nxt = run(dev(p), dev(tokens), dev(parents), dev(u), dev(ul), dev(q), None if tree_len is None else i32(tree_len))
    return run, path.cpu().numpy(), n.cpu().numpy(), nxt.cpu().numpy()


def check(p, q, tokens, parents, u, ul, path, n, nxt, tree_len=None):
    """Equality with the 64-bit rule wherever it has one answer: comparisons nearer than 2^-40 are beyond 48 bits."""
    B, T, V = p.shape
    told = 0
    for b in range(B):
        t = T if tree_len is None else tree_len[b]
        if t == 0:
            assert n[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            told += 1
            continue
        want, token, near = ref.verify(p[b, :t].astype(np.float64), None if q is None else q[b, :t].astype(np.float64), tokens[b, :t],
                                       parents[b, :t], u[b], ul[b])
        if near < 2.0 ** -40:
            continue
        told += 1
        assert n[b] == len(want) and list(path[b, :n[b]]) == want and (path[b, n[b]:] == -1).all(), b
        assert nxt[b] == token, b
    assert told >= B * 0.99


VERIFY = [
    # B, T, V, tree
    (1, 1, 1, "chain"),
    (3, 1, 1000, "chain"),
    (2, 2, 2, "chain"),
    (40, 6, 5, "chain"),
    (60, 4, 7, "wide"),
    (50, 9, 131, "random"),
    (9, 64, 257, "random"),
    (4, 12, 1027, "wide"),
    (3, 5, 50001, "chain"),
    (2, 8, 151936 // 2 + 1, "random"),
    (2, 3, 262144, "wide"),
]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,T,V,kind", VERIFY)
def test_verify(B, T, V, kind, drawn):
    a = trees(np.random.default_rng(B * T + V), B, T, V, kind, drawn)
    run, *got = call(*a)
    assert run.device_status() == 0
    check(*a, *got)


def test_every_outcome_occurs():
    """Among many small trees: all accepted, none accepted, rejected siblings before an accepted one, the last token drawn."""
    a = trees(np.random.default_rng(1), 4000, 5, 6, "random", True, spread=1.0)
    run, path, n, nxt = call(*a)
    check(*a, path, n, nxt)
    assert (n == 1).any() and (n == 5).any() and (n == 3).any() and set(nxt) == set(range(6))


def test_trees_of_different_lengths():
    a = trees(np.random.default_rng(2), 6, 10, 301, "random", True)
    tl = [10, 0, 1, 5, 0, 9]
    run, *got = call(*a, tree_len=tl)
    assert run.device_status() == 0
    check(*a, *got, tree_len=tl)


def test_certain_and_impossible_drafts():
    """p = q (every draft accepted), a draft that the target rules out, the same token drafted twice, u = 0, rows of zeros,
    values that are no probabilities."""
    V, T = 9, 3
    p = np.full((8, T, V), 1.0 / V, np.float32)
    q = p.copy()
    parents = np.tile(np.array([-1, 0, 1], np.int32), (8, 1))
    tokens = np.tile(np.array([0, 4, 7], np.int32), (8, 1))
    u, ul = np.full((8, T), 0.999999, np.float32), np.full(8, 0.5, np.float32)
    p[1, 0, 4] = 0.0  # sequence 1: the first draft is impossible
    parents[2] = [-1, 0, 0]  # 2: one token drafted twice below node 0, never accepted
    tokens[2] = [0, 4, 4]
    p[2, 0, 4] = 0.01
    p[3, 2] = 0.0  # 3: nothing after the last node
    p[4, 0] = [0, 0, 0, 0, 1, 0, 0, 0, 0]  # 4: the target is certain
    q[4, 0] = [0, 0, 0, 0, 1, 0, 0, 0, 0]
    p[5, 2, :4] = [math.nan, -1.0, math.inf, -math.inf]  # 5: count as 0
    u[6], ul[6] = 0.0, 0.0
    ul[7] = 2.0  # as the largest number below 1
    run, path, n, nxt = call(p, q, tokens, parents, u, ul)
    assert run.device_status() == 0
    assert list(n) == [3, 1, 1, 3, 3, 3, 3, 3]
    assert nxt[0] == 4 and nxt[3] == -1 and nxt[5] == 6 and nxt[6] == 0 and nxt[7] == V - 1
    # 1, 2: p is nowhere above q, so nothing is left and p itself is drawn from.  1: eight equal values, token 4 none: half of
    # their sum is not exceeded by tokens 0 .. 3, token 5 is the next.  2: the sum is 8/9 + 0.01, half of it 0.4494; tokens
    # 0 .. 3 hold 0.4444, 0 .. 4 hold 0.4544.
    assert nxt[1] == 5 and nxt[2] == 4
    run, path, n, nxt = call(p, None, tokens, parents, u, ul)
    assert list(n[[0, 1, 2, 4, 6]]) == [1, 1, 1, 2, 3] and nxt[0] != 4 and nxt[1] != 4 and nxt[2] != 4


def test_nothing_left_falls_back_to_the_target():
    """p below q everywhere but where both are 0 (rows that are no distributions): nothing is left of r."""
    p, q = np.full((1, 2, 4), 0.1, np.float32), np.full((1, 2, 4), 0.25, np.float32)
    run, path, n, nxt = call(p, q, np.array([[0, 1]], np.int32), np.array([[-1, 0]], np.int32), np.array([[0, 0.9]], np.float32),
                             np.array([0.6], np.float32))
    assert n[0] == 1 and nxt[0] == 2


@pytest.mark.parametrize("B", [3, 700])
def test_bad_parents_tokens_and_lengths(B):
    from block_sparse_long_index_gb300 import msa
    T, V = 16, 50
    a = list(trees(np.random.default_rng(3), B, T, V, "random", True))
    tl = [T] * B
    good = call(*a, tree_len=tl)[1:]
    for change in ("parent", "token", "long", "short"):
        tokens, parents, lens = a[2].copy(), a[3].copy(), list(tl)
        if change == "parent":
            parents[1, 5] = 5
        elif change == "token":
            tokens[1, 5] = V
        else:
            lens[1] = T + 1 if change == "long" else -1
        run, path, n, nxt = call(a[0], a[1], tokens, parents, a[4], a[5], lens)
        assert run.device_status() == msa.MSA_ERR_BAD_INDEX, change
        keep = np.arange(B) != 1
        assert all((x[keep] == y[keep]).all() for x, y in zip((path, n, nxt), good))
        if change in ("parent", "token"):
            assert 5 not in path[1] and n[1] >= 1 and 0 <= nxt[1] < V
        else:
            assert n[1] == 0 and nxt[1] == -1
    run, *_ = call(*a, run=run)
    assert run.device_status() == 0


def test_verify_stream_graph_and_refusals():
    from block_sparse_long_index_gb300 import DraftVerifier
    a = trees(np.random.default_rng(4), 5, 7, 333, "random", True)
    b = trees(np.random.default_rng(5), 5, 7, 333, "random", True)
    dev = [torch.tensor(x, device="cuda") for x in a]
    p, q, tok, par, u, ul = dev
    run, s = DraftVerifier(5, 7, 333), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(p, tok, par, u, ul, q, stream=s)
    s.synchronize()
    check(*a, run.path.cpu().numpy(), run.n_path.cpu().numpy(), run.next_token.cpu().numpy())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(p, tok, par, u, ul, q)
    for t, x in zip(dev, b):
        t.copy_(torch.tensor(x))
    g.replay()
    torch.cuda.synchronize()
    check(*b, run.path.cpu().numpy(), run.n_path.cpu().numpy(), run.next_token.cpu().numpy())
    for bad in (dict(probs=p[:4]), dict(probs=p.double()), dict(tokens=tok.long()), dict(parents=par[:, :3]), dict(u=u.cpu()), dict(u_last=ul[:2]),
                dict(draft_probs=q.half()), dict(tree_len=i32([1]))):
        with pytest.raises(ValueError):
            run(**{**dict(probs=p, tokens=tok, parents=par, u=u, u_last=ul), **bad})


# ---------------------------------------------------------------- the accepted branch
def cache_of(lens, page, n_pages, pools, seed=0):
    """A cache whose sequences have `lens` tokens, with marked rows in every pool, and each one's rows as numbers."""
    from block_sparse_long_index_gb300 import PagedCache
    B = len(lens)
    cache = PagedCache.empty(B, max(-(-n // page) for n in lens) + 1, n_pages, page, pools)
    order = np.random.default_rng(seed).permutation(B).tolist()
    cache.reserve(i32(order), i32([lens[s] for s in order]))
    assert cache.device_status() == 0
    for i, t in enumerate(pools):  # every row other than all others
        flat = t.view(torch.uint8).reshape(n_pages * page, -1)
        mark = torch.arange(n_pages * page, device="cuda")
        w = flat.shape[1]
        for j in range(w):
            flat[:, j] = (mark * (2 * j + 3) + (mark >> 8) * 7 + i * 11 + j).to(torch.uint8)
    return cache


def token_rows(cache, pool, s, n):
    t = cache.page_table[s].long()
    at = torch.arange(n, device="cuda")
    return pool.view(torch.uint8).reshape(cache.n_pages * cache.page_size, -1)[t[at // cache.page_size] * cache.page_size + at % cache.page_size].cpu()


POOLS = {
    "wide": lambda n, p: [torch.zeros((n, p, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)],
    "kv4": lambda n, p: [torch.zeros((n, p, 3, last), dtype=torch.uint8, device="cuda") for last in (32, 4, 32, 4)],
    "bytes": lambda n, p: [torch.zeros((n, p, 3), dtype=torch.uint8, device="cuda"), torch.zeros((n, p, 20), dtype=torch.uint8, device="cuda")],
    "many": lambda n, p: [torch.zeros((n, p, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(8)],
    "none": lambda n, p: [],
}


@pytest.mark.parametrize("kind", list(POOLS))
@pytest.mark.parametrize("page,T", [(16, 5), (64, 64), (32, 40)])
def test_accept(kind, page, T):
    r = np.random.default_rng(page + T)
    B = 7
    base = [0, 1, page - 1, page, 3 * page + 5, 2 * page - T % page, 100]
    extra = [T, T, T, T, T, T, T + 9]  # (the last one has tokens past its tree)
    lens = [b + e for b, e in zip(base, extra)]
    n_pages = sum(-(-n // page) for n in lens) + 5
    pools = POOLS[kind](n_pages, page)
    cache = cache_of(lens, page, n_pages, pools)
    paths = [sorted(r.choice(T, size=k, replace=False).tolist()) for k in (0, 1, T, T // 2, T // 3 + 1, 2, T - 1)]
    entries = [6, 2, 0, 5, 1, 3]  # 4 is not named
    before = [[token_rows(cache, p, s, lens[s]) for p in pools] for s in range(B)]
    old = [cache.page_table[s].clone() for s in range(B)]
    path = np.full((len(entries), T), -1, np.int32)
    for i, s in enumerate(entries):
        path[i, :len(paths[s])] = paths[s]
    cache.accept(i32(entries), i32([base[s] for s in entries]), i32(path), i32([len(paths[s]) for s in entries]))
    assert cache.device_status() == 0
    live = set()
    for s in range(B):
        n = base[s] + len(paths[s]) if s in entries else lens[s]
        held = -(-n // page)
        assert int(cache.ctx_len[s]) == n
        assert torch.equal(cache.page_table[s, :held], old[s][:held]) and bool((cache.page_table[s, held:] == -1).all())
        live |= set(old[s][:held].tolist())
        for p, was in zip(pools, before[s]):
            want = ref.accept(list(was), base[s], paths[s]) if s in entries else list(was)
            got = token_rows(cache, p, s, n)
            assert n == 0 or torch.equal(got, torch.stack(want))
    refs = cache.refs.cpu().numpy()
    assert all(refs[i] == (1 if i in live else 0) for i in range(n_pages))


def test_accept_changes_nothing_where_an_entry_is_bad():
    from block_sparse_long_index_gb300 import msa
    page, T, lens = 16, 4, [20, 40, 36]
    pools = POOLS["wide"](20, page)
    cache = cache_of(lens, page, 20, pools)
    good = dict(seqs=[0, 1], base=[16, 33], path=[[0, 2, -1, -1], [1, 3, 5, -1]], n_path=[2, 3])
    state = lambda: [t.view(torch.uint8) for t in (cache.page_table, cache.ctx_len, cache.refs, *pools)]  # noqa: E731  (some rows are NaN)
    keep = [t.clone() for t in state()]
    for bad in (dict(seqs=[0, 3]), dict(seqs=[-1, 1]), dict(seqs=[1, 1]), dict(base=[16, 41]), dict(base=[-1, 33]), dict(n_path=[2, 5]), dict(n_path=[2, -1]),
                dict(path=[[0, 2, -1, -1], [1, 3, 7, -1]]), dict(path=[[0, 2, -1, -1], [1, 1, 5, -1]]), dict(path=[[2, 0, -1, -1], [1, 3, 5, -1]]),
                dict(path=[[-1, 2, -1, -1], [1, 3, 5, -1]])):
        a = {**good, **bad}
        cache.accept(i32(a["seqs"]), i32(a["base"]), i32(a["path"]), i32(a["n_path"]))
        assert cache.device_status() == msa.MSA_ERR_BAD_INDEX, bad
        assert all(torch.equal(x, y) for x, y in zip(keep, state())), bad
    cache.refs[cache.page_table[1, 2].long()] = 2  # a page from base on that another sequence holds too
    cache.accept(*[i32(good[n]) for n in ("seqs", "base", "path", "n_path")])
    assert cache.device_status() == msa.MSA_ERR_BAD_INDEX and int(cache.ctx_len[0]) == 20
    cache.refs[cache.page_table[1, 2].long()] = 1
    cache.refs[cache.page_table[1, 1].long()] = 2  # one before it may be shared
    cache.accept(*[i32(good[n]) for n in ("seqs", "base", "path", "n_path")])
    assert cache.device_status() == 0 and cache.ctx_len.tolist() == [18, 36, 36]
    many = i32([0] * 50)  # more entries than sequences: one is named twice
    cache.accept(many, many, i32([[0]] * 50), many)
    assert cache.device_status() == msa.MSA_ERR_BAD_INDEX and cache.ctx_len.tolist() == [18, 36, 36]
    cache.accept(i32([]), i32([]), i32(np.zeros((0, 3))), i32([]))
    assert cache.device_status() == 0
    for bad in (lambda: cache.accept(i32([0]), i32([0, 1]), i32([[0]]), i32([1])), lambda: cache.accept(i32([0]), i32([0]), i32([[0]]).long(), i32([1]))):
        with pytest.raises(ValueError):
            bad()


def test_a_shared_prefix_is_kept():
    """After a fork both samples speculate: the shared full pages stay shared, each one's own branch goes its way."""
    page, pools = 16, POOLS["wide"](12, 16)
    cache = cache_of([37, 1], page, 12, pools)
    cache.free(i32([1]))
    cache.fork(i32([0]), i32([1]))
    cache.reserve(i32([0, 1]), i32([37 + 6, 37 + 6]))
    assert cache.device_status() == 0
    before = [token_rows(cache, pools[0], s, 43) for s in (0, 1)]
    cache.accept(i32([0, 1]), i32([37, 37]), i32([[0, 1, 4], [0, 5, -1]]), i32([3, 2]))
    assert cache.device_status() == 0 and cache.ctx_len.tolist() == [40, 39]
    assert torch.equal(cache.page_table[0, :2], cache.page_table[1, :2]) and cache.refs[cache.page_table[0, 0].long()] == 2
    for s, path in ((0, [0, 1, 4]), (1, [0, 5])):
        assert torch.equal(token_rows(cache, pools[0], s, 37 + len(path)), torch.stack(ref.accept(list(before[s]), 37, path)))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_speculative_run(kind):
    """Steps of a speculative decode on one layer: drafts appended at their depths, attended, verified, kept.  Afterwards the
    cache holds what appending the accepted tokens one after the other would have left, bit for bit, and attention over it
    is that of the accepted nodes."""
    from block_sparse_long_index_gb300 import DraftVerifier, Kv4Pool, KvPool, MsaTreeDecode, PagedCache, Rope
    r = np.random.default_rng(7)
    B, T, H_q, H_kv, d, d_I, V, page, n_pages = 3, 6, 8, 2, 64, 32, 40, 16, 64
    make = KvPool if kind == "bf16" else Kv4Pool
    pool, plain = make.empty(n_pages, page, H_kv, d), make.empty(n_pages, page, H_kv, d)
    idx = [torch.zeros((n_pages, page, d_I), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = PagedCache.empty(B, 8, n_pages, page, pool.tensors() + [idx[0]])
    rope, idx_rope = Rope(32), Rope(16, interleaved=True)
    table_k, table_v = rows(V, H_kv, d, seed=1), rows(V, H_kv, d, seed=2)  # a "model": rows by token
    table_q, table_i = rows(V, H_q, d, seed=3), rows(V, d_I, seed=4)
    ctx = [5, 0, 17]
    text = [r.integers(0, V, n).tolist() for n in ctx]
    cu = lambda n: i32([sum(n[:i]) for i in range(len(n) + 1)])  # noqa: E731
    cache.reserve(i32(range(B)), i32(ctx))
    flat = torch.tensor(sum(text, []), device="cuda", dtype=torch.long)
    pool.append(table_k[flat], table_v[flat], cu(ctx), i32([0] * B), cache.page_table, rope=rope, k_idx=table_i[flat], k_idx_pool=idx[0],
                idx_rope=idx_rope)
    last = r.integers(0, V, B).tolist()  # the token that each step begins with
    dec, ver, graph = MsaTreeDecode(pool, B, T, 8, H_q), DraftVerifier(B, T, V), None
    for step in range(6):
        parents = np.array([ref.tree_of(r, T, ["random", "chain", "wide"][(step + b) % 3]) for b in range(B)], np.int32)
        depth = np.array([[len(line) - 1 for line in ref.ancestors(par)] for par in parents])
        tokens = r.integers(0, V, (B, T)).astype(np.int32)
        tokens[:, 0] = last
        base = i32([len(t) for t in text])
        cache.reserve(i32(range(B)), base + T)
        x = torch.tensor(tokens.reshape(-1), device="cuda", dtype=torch.long)
        pos = (base[:, None] + i32(depth)).flatten().contiguous()
        q, _ = pool.append(table_k[x], table_v[x], cu([T] * B), base, cache.page_table, rope=rope, positions=pos, q=table_q[x],
                           k_idx=table_i[x], k_idx_pool=idx[0], idx_rope=idx_rope)
        assert pool.device_status() == 0
        out, lse = dec(q.unflatten(0, (B, T)), cache.page_table, base, i32(parents))
        assert dec.device_status() == 0
        # a target that depends on what was attended, sharp enough that some drafts are accepted
        w = rows(H_q * d, V, seed=5, dtype=torch.float32, scale=0.3)
        logits = out.float().flatten(2) @ w
        logits.scatter_add_(2, torch.tensor(np.roll(tokens, -1, 1), device="cuda", dtype=torch.long)[..., None], torch.full((B, T, 1), 4.0, device="cuda"))
        p = torch.softmax(logits, -1).contiguous()
        u, ul = (torch.tensor(r.random(s), device="cuda", dtype=torch.float32) for s in ((B, T), (B,)))
        path, n_path, nxt = ver(p, i32(tokens), i32(parents), u, ul)
        attended, first = out.clone(), base.tolist()
        cache.accept(i32(range(B)), base, path, n_path)
        assert cache.device_status() == 0 and ver.device_status() == 0
        for b in range(B):
            line = path[b, :int(n_path[b])].tolist()
            text[b] += [int(tokens[b, j]) for j in line]
            if step == 3:  # the accepted nodes, attended again one by one, as single tokens of the kept cache
                one = MsaTreeDecode(pool, 1, 1, 8, H_q)
                for i, j in enumerate(line):
                    o, _ = one(q.unflatten(0, (B, T))[b:b + 1, j:j + 1].contiguous(), cache.page_table[b:b + 1], i32([first[b] + i]), i32([[-1]]))
                    assert float((o[0, 0].float() - attended[b, j].float()).abs().max()) < 0.03
        last = nxt.tolist()
        assert cache.ctx_len.tolist() == [len(t) for t in text]
    lens = [len(t) for t in text]
    assert max(lens) > max(ctx) + 6  # drafts were accepted
    flat = torch.tensor(sum(text, []), device="cuda", dtype=torch.long)
    plain.append(table_k[flat], table_v[flat], cu(lens), i32([0] * B), cache.page_table, rope=rope, k_idx=table_i[flat], k_idx_pool=idx[1],
                 idx_rope=idx_rope)
    for got, want in zip(pool.tensors() + [idx[0]], plain.tensors() + [idx[1]]):
        for b in range(B):
            assert torch.equal(token_rows(cache, got, b, lens[b]), token_rows(cache, want, b, lens[b]))


def test_speculative_step_captured():
    """Append, attend, verify and accept in one graph, replayed step after step with new inputs."""
    from block_sparse_long_index_gb300 import DraftVerifier, KvPool, MsaTreeDecode, PagedCache, Rope
    B, T, H_q, H_kv, d, V, page, n_pages = 2, 4, 4, 2, 64, 100, 16, 32
    rope, cu = Rope(64), i32([0, T, 2 * T])

    def fresh():
        pool = KvPool.empty(n_pages, page, H_kv, d)
        cache = PagedCache.empty(B, 8, n_pages, page, pool.tensors())
        cache.reserve(i32([0, 1]), i32([9, 30]))
        for i, t in enumerate(pool.tensors()):
            t.copy_(rows(*t.shape, seed=50 + i))
        return pool, cache, MsaTreeDecode(pool, B, T, 8, H_q), DraftVerifier(B, T, V), torch.tensor([9, 30], dtype=torch.int32, device="cuda")

    x = dict(k=rows(B * T, H_kv, d), v=rows(B * T, H_kv, d), q=rows(B * T, H_q, d), p=torch.empty((B, T, V), device="cuda"),
             tokens=torch.zeros((B, T), dtype=torch.int32, device="cuda"), parents=torch.zeros((B, T), dtype=torch.int32, device="cuda"),
             depth=torch.zeros((B, T), dtype=torch.int32, device="cuda"), u=torch.zeros((B, T), device="cuda"), ul=torch.zeros(B, device="cuda"))
    seqs = i32([0, 1])

    def step(pool, cache, dec, ver, base):
        cache.reserve(seqs, base + T)
        q, _ = pool.append(x["k"], x["v"], cu, base, cache.page_table, rope=rope, positions=(base[:, None] + x["depth"]).flatten(), q=x["q"])
        dec(q.unflatten(0, (B, T)), cache.page_table, base, x["parents"])
        path, n_path, _ = ver(x["p"], x["tokens"], x["parents"], x["u"], x["ul"])
        cache.accept(seqs, base, path, n_path)
        base.add_(n_path)

    def load(i):
        r = np.random.default_rng(i)
        par = np.array([ref.tree_of(r, T, "random") for _ in range(B)], np.int32)
        new = dict(k=rows(B * T, H_kv, d, seed=i), v=rows(B * T, H_kv, d, seed=i + 100), q=rows(B * T, H_q, d, seed=i + 200),
                   p=torch.softmax(rows(B, T, V, dtype=torch.float32, seed=i, scale=3.0), -1), tokens=i32(r.integers(0, 8, (B, T))),
                   parents=i32(par), depth=i32([[len(y) - 1 for y in ref.ancestors(z)] for z in par]),
                   u=torch.tensor(r.random((B, T)) * 0.02, device="cuda", dtype=torch.float32), ul=torch.tensor(r.random(B), device="cuda", dtype=torch.float32))
        for n, t in new.items():
            x[n].copy_(t)

    eager, replayed = fresh(), fresh()
    load(0)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        step(*replayed)
    for i in range(1, 6):
        load(i)
        step(*eager)
        g.replay()
        torch.cuda.synchronize()
        assert all(a.device_status() == 0 for a in (*eager[:4], *replayed[:4]))
        for a, b in zip(eager[0].tensors() + [eager[1].page_table, eager[1].ctx_len, eager[1].refs, eager[2].out, eager[3].path, eager[4]],
                        replayed[0].tensors() + [replayed[1].page_table, replayed[1].ctx_len, replayed[1].refs, replayed[2].out, replayed[3].path, replayed[4]]):
            assert torch.equal(a, b)
    assert int(eager[4].sum()) > 39 + 10


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,T,V,kind", [(24, 4, 9001, "random"), (45, 5, 7003, "random"), (41, 1, 20000, "chain")])
def test_verify_many_trees_over_long_rows(B, T, V, kind, drawn):
    a = trees(np.random.default_rng(B + V), B, T, V, kind, drawn)
    run, *got = call(*a)
    assert run.device_status() == 0
    check(*a, *got)


def many_accepts(n=150, T=30, page=16, seed=31):
    """More entries than the plan's first form takes: random bases and branches, sequences of 0 to 200 tokens before them."""
    r = np.random.default_rng(seed)
    base = r.integers(0, 200, n)
    base[:4] = [0, page, page - 1, 1]
    lens = [int(b) + T + int(e) for b, e in zip(base, r.integers(0, 20, n))]
    n_pages = sum(-(-x // page) for x in lens) + 5
    pools = [torch.zeros((n_pages, page, 2, 8), dtype=torch.bfloat16, device="cuda")]
    cache = cache_of(lens, page, n_pages, pools, seed=seed)
    k = r.integers(0, T + 1, n)
    k[:6] = [0, T, 1, T - 1, 0, T]
    paths = [sorted(r.choice(T, size=x, replace=False).tolist()) for x in k]
    entries = r.permutation(n)[:n - 7]
    path = np.full((len(entries), T), -1, np.int32)
    for i, s in enumerate(entries):
        path[i, :k[s]] = paths[s]
    return cache, pools, lens, base, paths, entries, path


def test_accept_of_many_entries():
    cache, pools, lens, base, paths, entries, path = many_accepts()
    page = cache.page_size
    before = [token_rows(cache, pools[0], s, n) for s, n in enumerate(lens)]
    old = cache.page_table.clone()
    cache.accept(i32(entries), i32(base[entries]), i32(path), i32([len(paths[s]) for s in entries]))
    assert cache.device_status() == 0
    live = set()
    for s, n0 in enumerate(lens):
        named = s in entries
        n = int(base[s]) + len(paths[s]) if named else n0
        held = -(-n // page)
        assert int(cache.ctx_len[s]) == n
        assert torch.equal(cache.page_table[s, :held], old[s, :held]) and bool((cache.page_table[s, held:] == -1).all())
        live |= set(old[s, :held].tolist())
        want = ref.accept(list(before[s]), int(base[s]), paths[s]) if named else list(before[s])
        assert n == 0 or torch.equal(token_rows(cache, pools[0], s, n), torch.stack(want))
    refs = cache.refs.cpu().numpy()
    assert all(refs[i] == (1 if i in live else 0) for i in range(cache.n_pages))


@pytest.mark.parametrize("what", ["a name twice", "a name outside", "a base past the end", "a path that falls", "a node past the end", "a shared page"])
def test_accept_of_many_entries_changes_nothing_where_one_is_bad(what):
    from block_sparse_long_index_gb300 import msa
    cache, pools, lens, base, paths, entries, path = many_accepts(seed=32)
    seqs, bases, n = entries.copy(), base[entries].copy(), np.array([len(paths[s]) for s in entries])
    at = next(i for i in range(100, len(seqs)) if n[i] > 3)
    if what == "a name twice":
        seqs[at] = seqs[3]
        bases[at], n[at] = 0, 0
    elif what == "a name outside":
        seqs[at] = len(lens)
    elif what == "a base past the end":
        bases[at], n[at] = lens[seqs[at]] + 1, 0
    elif what == "a path that falls":
        path[at, 2] = path[at, 1]
    elif what == "a node past the end":
        path[at, n[at] - 1] = lens[seqs[at]] - bases[at]
    else:
        cache.refs[cache.page_table[seqs[at], int(bases[at]) // 16].long()] = 2
    held = (cache.page_table, cache.ctx_len, cache.refs, pools[0].view(torch.uint8))  # (the rows' bytes make NaNs, too)
    state = [t.clone() for t in held]
    cache.accept(i32(seqs), i32(bases), i32(path), i32(n))
    assert cache.device_status() == msa.MSA_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(state, held))
