"""The calls of a speculative decode step at the largest sizes that they take."""
import math

import numpy as np
import pytest
import torch

import serving_ref as sref
from test_gpu_kv4 import i32
from test_gpu_rope import rows

pytestmark = pytest.mark.gpu


def test_verify_the_longest_vocabulary():
    from block_sparse_long_index_gb300 import DraftVerifier
    V = (1 << 31) - 1
    p = torch.zeros((1, 1, V), device="cuda")
    places = [0, (1 << 30) + 1, V - 1]
    p[0, 0, places] = torch.tensor([0.25, 0.25, 0.5], device="cuda")
    run, zero, f32 = DraftVerifier(1, 1, V), i32([[0]]), lambda x: torch.tensor(x, device="cuda")
    for u, want in ((0.2, 0), (0.25, 1), (0.4, 1), (0.6, 2), (2.0, 2)):  # (u times the sum is exceeded: 0.25 is not by 0.25)
        _, n, token = run(p, zero, i32([[-1]]), f32([[0.5]]), f32([u]))
        assert run.device_status() == 0 and int(n) == 1 and int(token) == places[want]


def test_verify_the_most_trees():
    from block_sparse_long_index_gb300 import DraftVerifier
    B, V = 1 << 20, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.softmax(torch.randn((B, 2, V), generator=g, device="cuda"), -1)
    u, ul = torch.rand((B, 2), generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    tokens = torch.randint(0, V, (B, 2), generator=g, device="cuda").int()
    run = DraftVerifier(B, 2, V)
    path, n, token = run(p, tokens, i32([[-1, 0]]).expand(B, 2).contiguous(), u, ul)
    assert run.device_status() == 0
    x = tokens[:, 1].long()
    lhs, rhs = u[:, 1].double(), p[torch.arange(B, device="cuda"), 0, x].double()  # certain drafts: accepted where u < p(x)
    yes = lhs < rhs
    r = torch.where(yes[:, None], p[:, 1], p[:, 0].scatter(1, x[:, None], 0.0)).double()
    r[yes] = p[yes, 1].double()
    cum = r.cumsum(1)
    at = ul.double() * cum[:, -1]
    sure = ((cum - at[:, None]).abs().amin(1) > 2.0 ** -40) & ((lhs - rhs).abs() > 2.0 ** -40)
    assert int(sure.sum()) > B * 0.999
    want = (cum <= at[:, None]).sum(1).int()
    assert torch.equal(n[sure], (1 + yes.int())[sure].int()) and torch.equal(token[sure], want[sure])
    assert torch.equal(path[sure, 1], torch.where(yes, 1, -1).int()[sure])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_the_most_trees(kind):
    """2^20 sequences that all read the same few pages, one node each."""
    from block_sparse_long_index_gb300 import Kv4Pool, KvPool, MsaTreeDecode
    B, d, page, n_pages = 1 << 20, 64, 16, 7
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = rows(n_pages * page, 1, d, seed=3), rows(n_pages * page, 1, d, seed=4)
    pool = (KvPool if kind == "bf16" else Kv4Pool).empty(n_pages, page, 1, d)
    at = (i32([0, n_pages * page]), i32([0]), i32([list(range(n_pages))]))
    pool.append(k, v, *at)
    if kind == "kv4":
        k, v = pool.load(n_pages * page, *at)
    q = rows(B, 1, 1, d, seed=5)
    table = torch.randint(0, n_pages, (B, 1), generator=g, device="cuda").int()
    ctx = torch.randint(0, page, (B,), generator=g, device="cuda").int()
    dec = MsaTreeDecode(pool, B, 1, 1, 1)
    out, lse = dec(q, table, ctx, torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), scale=0.125)
    assert dec.device_status() == 0
    some = torch.cat([torch.arange(3, device="cuda"), torch.randint(0, B, (5000,), generator=g, device="cuda"), torch.arange(B - 3, B, device="cuda")])
    kk, vv = (x.view(n_pages, page, d)[table[some, 0].long()].double() for x in (k, v))
    hidden = torch.arange(page, device="cuda") > ctx[some, None]
    qq = q[some, 0, 0].double()
    x = (torch.einsum("bd,bnd->bn", qq, kk) * 0.125).masked_fill_(hidden, -math.inf)
    p = torch.softmax(x, -1)
    S = torch.einsum("bd,bnd->bn", qq.abs(), kk.abs()).masked_fill_(hidden, 0.0).amax(-1) * 0.125
    sref.check_attention(out[some, 0, 0], lse[some, 0, 0], torch.einsum("bn,bnd->bd", p, vv), torch.logsumexp(x, -1),
                         torch.einsum("bn,bnd->bd", p, vv.abs()), S, d, page)


def test_accept_the_most_entries():
    from block_sparse_long_index_gb300 import PagedCache
    r = np.random.default_rng(6)
    n, T, page = 4096, 64, 16
    base = r.integers(0, 50, n)
    lens = base + T
    n_pages = int(sum(-(-lens // page))) + 3
    pool = torch.arange(n_pages * page * 4, device="cuda", dtype=torch.int32).view(n_pages, page, 4)  # every row other than all others
    cache = PagedCache.empty(n, 8, n_pages, page, [pool])
    cache.reserve(i32(np.arange(n)), i32(lens))
    assert cache.device_status() == 0
    k = r.integers(0, T + 1, n)
    path = np.full((n, T), -1, np.int64)
    for i in range(n):
        path[i, :k[i]] = np.sort(r.permutation(T)[:k[i]])
    table, was, order = cache.page_table.cpu().numpy().astype(np.int64), pool.cpu().numpy().reshape(-1, 4).copy(), r.permutation(n)
    cache.accept(i32(order), i32(base[order]), i32(path[order]), i32(k[order]))
    assert cache.device_status() == 0
    seq, j = np.nonzero(np.arange(T) < k[:, None])
    row = lambda t: table[seq, t // page] * page + t % page  # noqa: E731
    src, dst = row(base[seq] + path[seq, j]), row(base[seq] + j)
    want = was.copy()
    want[dst] = was[src]
    assert (pool.cpu().numpy().reshape(-1, 4) == want).all()
    end = base + k
    held = -(-end // page)
    assert (cache.ctx_len.cpu().numpy() == end).all()
    assert (cache.page_table.cpu().numpy() == np.where(np.arange(8) < held[:, None], table, -1)).all()
    assert int(cache.refs.sum()) == int(held.sum())
