"""Page tables on the GPU against plain lists, and a serving run of the operators together."""
import math
import random

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Both:
    """A PagedCache and the plain one, with page contents that name their origin."""

    def __init__(self, n_seqs, max_pages, n_pages, page):
        from block_sparse_long_index_gb300 import PagedCache
        ids = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.pools = [ids[:, None, None].expand(n_pages, page, 4).contiguous(),
                      ids[:, None].to(torch.int16).expand(n_pages, page).contiguous(),
                      ids[:, None, None].to(torch.uint8).expand(n_pages, page, 1100).contiguous()]
        self.gpu = PagedCache.empty(n_seqs, max_pages, n_pages, page, self.pools)
        self.ref = ref.PagesRef(n_seqs, max_pages, n_pages, page)

    def check(self):
        assert self.gpu.ctx_len.tolist() == self.ref.ctx
        assert self.gpu.refs.tolist() == self.ref.refs
        for row, want in zip(self.gpu.page_table.tolist(), self.ref.table):
            assert row[:len(want)] == want
        data = torch.tensor(self.ref.data, dtype=torch.int32, device="cuda")
        for p in self.pools:
            assert bool((p == data.to(p.dtype).view(-1, *[1] * (p.dim() - 1))).all())


@pytest.mark.parametrize("seed,n_seqs,n_pages,page", [(0, 6, 40, 16), (1, 20, 300, 32), (2, 3, 9, 16), (3, 50, 5000, 16)])
def test_against_lists(seed, n_seqs, n_pages, page):
    """Random reserves, forks, frees and compactions, with the state compared after each."""
    r = random.Random(seed)
    most = max(2, 2 * n_pages // n_seqs)
    b = Both(n_seqs, most, n_pages, page)
    from block_sparse_long_index_gb300 import msa
    refused = 0
    for _ in range(40):
        what = r.choice(["reserve", "reserve", "fork", "free", "compact"])
        empty = [s for s in range(n_seqs) if b.ref.ctx[s] == 0]
        if what == "reserve":
            seqs = r.sample(range(n_seqs), r.randint(1, n_seqs))
            lens = [r.randint(b.ref.ctx[s], min(most * page, b.ref.ctx[s] + r.choice([1, page, 5 * page]))) for s in seqs]
            ok = b.ref.reserve(seqs, lens)
            b.gpu.reserve(i32(seqs), i32(lens))
        elif what == "fork" and empty:
            dst = r.sample(empty, r.randint(1, len(empty)))
            src = [r.randrange(n_seqs) for _ in dst]
            ok = b.ref.fork(src, dst)
            b.gpu.fork(i32(src), i32(dst))
        elif what == "free":
            seqs = [r.randrange(n_seqs) for _ in range(r.randint(1, 4))]  # a sequence may be named twice
            b.ref.free(seqs)
            ok = True
            b.gpu.free(i32(seqs))
        else:
            page_map, n_live = b.ref.compact()
            ok = True
            m, n = b.gpu.compact()
            assert m.tolist() == page_map and n.tolist() == [n_live]
        assert b.gpu.device_status() == (0 if ok else msa.MSA_ERR_NO_PAGES)
        refused += not ok
        b.check()


def test_no_entries_and_no_pools():
    from block_sparse_long_index_gb300 import PagedCache
    c = PagedCache.empty(2, 4, 8, 16)
    none = i32([])
    c.reserve(none, none)
    c.fork(none, none)
    c.free(none)
    c.reserve(i32([1]), i32([20]))
    m, n = c.compact()
    assert c.device_status() == 0 and n.tolist() == [2] and m.tolist() == [0, 1] + [-1] * 6


def test_refusals_change_nothing():
    from block_sparse_long_index_gb300 import msa
    b = Both(5, 3, 8, 16)
    b.ref.reserve([0, 1], [20, 48])
    b.gpu.reserve(i32([0, 1]), i32([20, 48]))
    b.check()
    for seqs, lens in (([5], [1]), ([-1], [1]), ([0], [19]), ([0], [49]), ([2, 2], [16, 16]), ([3, 0], [16, 3])):
        b.gpu.reserve(i32(seqs), i32(lens))
        assert b.gpu.device_status() == msa.MSA_ERR_BAD_INDEX, (seqs, lens)
        b.check()
    b.gpu.reserve(i32([2, 3]), i32([32, 32]))  # 4 pages, 3 free
    assert b.gpu.device_status() == msa.MSA_ERR_NO_PAGES
    b.check()
    for src, dst in (([0], [1]), ([0], [7]), ([9], [2]), ([0, 0], [2, 2])):
        b.gpu.fork(i32(src), i32(dst))
        assert b.gpu.device_status() == msa.MSA_ERR_BAD_INDEX, (src, dst)
        b.check()
    b.gpu.free(i32([-1, 0, 5]))  # the bad entries are passed over
    assert b.gpu.device_status() == msa.MSA_ERR_BAD_INDEX
    b.ref.free([0])
    b.check()
    b.gpu.page_table[1, 2] = 99
    b.gpu.free(i32([1]))
    assert b.gpu.device_status() == msa.MSA_ERR_BAD_INDEX
    assert b.gpu.ctx_len.tolist()[1] == 48 and b.gpu.refs.tolist() == b.ref.refs


def test_fork_of_a_fork_target():
    """An empty source that the same call also fills: it is forked as it was when the call began."""
    b = Both(4, 3, 8, 16)
    b.ref.reserve([0], [20])
    b.gpu.reserve(i32([0]), i32([20]))
    b.ref.fork([0, 1, 3], [1, 2, 3])
    b.gpu.fork(i32([0, 1, 3]), i32([1, 2, 3]))
    assert b.gpu.device_status() == 0
    b.check()
    assert b.ref.ctx == [20, 20, 0, 0]


def test_graph_replay():
    """A captured reserve-and-free cycle gives the same pages each time."""
    b = Both(3, 4, 10, 16)
    seqs, lens, to = i32([1]), i32([40]), i32([2])
    b.gpu.reserve(seqs, lens)
    b.gpu.free(seqs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.gpu.reserve(seqs, lens)
        b.gpu.fork(seqs, to)
    for _ in range(3):
        g.replay()
        b.gpu.free(i32([1, 2]))
        assert b.gpu.device_status() == 0
        assert b.gpu.refs.tolist() == [0] * 10
    g.replay()
    torch.cuda.synchronize()
    b.ref.reserve([1], [40])
    b.ref.fork([1], [2])
    b.check()


def test_serving_run():
    """Prompts prefilled together, stored in 4 bits, forked, extended token by token, some of them freed and the
    cache compacted: every decode step equals 64-bit attention over the history that the cache stands for."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4, MsaDensePrefill, PagedCache
    H_q, H_kv, d, d_I, page, n_pages, n_seqs = 8, 2, 64, 32, 16, 60, 6
    lens, scale = [37, 64, 5], 1 / math.sqrt(64)
    N = sum(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    pool = Kv4Pool.empty(n_pages, page, H_kv, d)
    k_idx = torch.zeros(n_pages, page, d_I, dtype=torch.bfloat16, device="cuda")
    cache = PagedCache.empty(n_seqs, 8, n_pages, page, pool.tensors() + [k_idx])
    # prefill and store
    q, k, v = rnd(N, H_q, d), rnd(N, H_kv, d), rnd(N, H_kv, d)
    cu = i32([0, 37, 101, 106])
    out, lse = MsaDensePrefill(N, H_q, H_kv, d, 3)(q, k, v, cu)
    ref.check_attention(out, lse.T, *ref.dense_prefill(q, k, v, lens, scale), d, 64)
    cache.reserve(i32([0, 1, 2]), i32(lens))
    pool.store(k, v, cu, i32([0, 0, 0]), cache.page_table[:3])
    k4, v4 = pool.load(N, cu, i32([0, 0, 0]), cache.page_table[:3])
    hist = {s: (k4[a:b], v4[a:b]) for s, (a, b) in enumerate(((0, 37), (37, 101), (101, 106)))}
    # two more samples of the first prompt and one of the second
    cache.fork(i32([0, 0, 1]), i32([3, 4, 5]))
    for s, t in ((0, 3), (0, 4), (1, 5)):
        hist[t] = hist[s]
    run = MsaDecodeKv4(pool, n_seqs, 8, H_q, d_I=d_I, Bk=64, k=2)
    ones = i32(range(n_seqs + 1))
    gone = []
    for step in range(20):
        live = [s for s in range(n_seqs) if s not in gone]
        before = cache.ctx_len.clone()
        cache.reserve(i32(live), i32([hist[s][0].shape[0] + 1 for s in live]))
        kt, vt = rnd(n_seqs, H_kv, d), rnd(n_seqs, H_kv, d)
        cu_t = ones if not gone else i32([sum(s in live for s in range(t)) for t in range(n_seqs + 1)])
        pool.store(kt[:len(live)], vt[:len(live)], cu_t, before, cache.page_table)
        ka, va = pool.load(len(live), cu_t, before, cache.page_table)
        for i, s in enumerate(live):
            hist[s] = (torch.cat([hist[s][0], ka[i:i + 1]]), torch.cat([hist[s][1], va[i:i + 1]]))
        qt = rnd(n_seqs, H_q, d)
        o, l = run.dense(qt, cache.page_table, cache.ctx_len, scale)
        assert run.device_status() == 0 and cache.device_status() == 0 and pool.device_status() == 0
        for s in live:
            parts = [ref.attend(qt[s, 4 * h:4 * h + 4].double(), hist[s][0][:, h].double(), hist[s][1][:, h].double(), scale)
                     for h in range(H_kv)]
            ro, rl, A, S = [torch.cat([p[i] for p in parts]) for i in range(4)]
            ref.check_attention(o[s], l[s], ro, rl, A, S, d, hist[s][0].shape[0])
        for s in gone:
            assert bool((o[s] == 0).all())
        if step == 9:
            gone = [0, 5]
            cache.free(i32(gone))
            _, n_live = cache.compact()
            assert int(n_live) == int((cache.refs > 0).sum()) and bool((cache.refs[:int(n_live)] > 0).all())
    # the MSA step over the same cache, every block chosen
    o2, l2, blk = run(qt, rnd(n_seqs, H_kv, d_I), k_idx, cache.page_table, cache.ctx_len.clamp(min=1), scale)
    for s in live:
        assert float((o2[s].float() - o[s].float()).norm() / o[s].float().norm()) < 2 * ref.BF16_HALF
