"""The serving classes together: what their calls return stays until its own buffer is written again, the MSA step after
a cache was forked, freed and compacted, page calls that refuse, calls at once, captured calls, and statuses."""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_dense_prefill import make
from test_gpu_kv4 import dense_ref, i32, random_pool, table_of

pytestmark = pytest.mark.gpu


def rnd(*s):
    return torch.randn(*s, device="cuda").to(torch.bfloat16)


def test_dense_and_step_keep_their_outputs():
    """One object's two operators have buffers of their own; out and lse are those of the last call."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    ctx, page, H_kv, d = [500, 130], 16, 2, 64
    counts = [-(-c // page) for c in ctx]
    pool, table = random_pool(sum(counts), page, H_kv, d), table_of(counts, max(counts), sum(counts))
    q, qi, ki = rnd(2, 8, d), rnd(2, H_kv, 64), rnd(sum(counts), page, 64)
    a, b = (MsaDecodeKv4(pool, 2, max(counts), 8, d_I=64, Bk=64, k=2) for _ in range(2))
    want = [t.clone() for t in b.dense(q, table, i32(ctx), 0.1)]
    step = [t.clone() for t in b(q, qi, ki, table, i32(ctx), 0.1)]
    assert not torch.equal(want[0], step[0])
    got = a.dense(q, table, i32(ctx), 0.1)
    assert a.out is got[0] and a.lse is got[1]
    got2 = a(q, qi, ki, table, i32(ctx), 0.1)
    assert a.out is got2[0] and a.lse is got2[1]
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and all(torch.equal(x, y) for x, y in zip(got2, step))
        a.dense(q, table, i32(ctx), 0.1)
    assert a.device_status() == 0 and b.device_status() == 0


def test_step_of_a_cache_that_was_forked_freed_and_compacted():
    """With every block chosen the MSA step is the dense step: compared with it, and with 64 bits, after the page calls
    have moved the sequences about."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4, PagedCache
    H_q, H_kv, d, d_I, page, n_pages, n_seqs, Bk, k = 8, 2, 64, 32, 16, 60, 6, 64, 3
    lens = [37, 150, 64]
    N = sum(lens)
    pool = Kv4Pool.empty(n_pages, page, H_kv, d)
    ki = torch.zeros(n_pages, page, d_I, dtype=torch.bfloat16, device="cuda")
    cache = PagedCache.empty(n_seqs, 12, n_pages, page, pool.tensors() + [ki])
    cache.reserve(i32([0, 1, 2]), i32(lens))
    pool.store(rnd(N, H_kv, d), rnd(N, H_kv, d), i32([0, 37, 187, 251]), i32([0, 0, 0]), cache.page_table[:3])
    ki.copy_(rnd(*ki.shape))
    cache.fork(i32([1, 0, 1]), i32([3, 4, 5]))
    before = cache.ctx_len.clone()
    cache.reserve(i32(range(n_seqs)), before + 1)
    pool.store(rnd(n_seqs, H_kv, d), rnd(n_seqs, H_kv, d), i32(range(n_seqs + 1)), before, cache.page_table)
    cache.free(i32([1, 4]))
    cache.compact()
    live = [0, 2, 3, 5]
    table, ctx = cache.page_table[live].contiguous(), cache.ctx_len[live].contiguous()
    n = ctx.tolist()
    assert cache.device_status() == 0 and pool.device_status() == 0 and n == [38, 65, 151, 151]
    q, qi = rnd(4, H_q, d), rnd(4, H_kv, d_I)
    run = MsaDecodeKv4(pool, 4, 12, H_q, d_I=d_I, Bk=Bk, k=k)
    o, l = run.dense(q, table, ctx, 0.125)
    assert run.device_status() == 0
    run._step[0].fill_(7.0)
    run._step[1].fill_(7.0)
    run.block_idx.fill_(99)
    o2, l2, blk = run(q, qi, ki, table, ctx, 0.125)
    assert run.device_status() == 0 and o2.data_ptr() != o.data_ptr()
    for b in range(4):
        nb = -(-n[b] // Bk)
        for g in range(H_kv):
            assert sorted(blk[b, g].tolist()) == [-1] * (k - nb) + list(range(nb))
    want = dense_ref(pool, q, table, n, 0.125)
    ref.check_attention(o, l, *want, d, max(n))
    ref.check_attention(o2, l2, *want, d, max(n))  # (the merge of k partials is an fp32 sum of k terms more)


# ---------------------------------------------------------------- pages
def tables(cache):
    return [t.clone() for t in [cache.page_table, cache.ctx_len, cache.refs] + cache.pools]


def test_more_entries_than_sequences():
    """Such a call names a sequence twice or one that is not there: the device says so, and nothing changes."""
    from block_sparse_long_index_gb300 import PagedCache, msa
    cache = PagedCache.empty(2, 4, 8, 16)
    cache.reserve(i32([0]), i32([20]))
    was = tables(cache)
    many = i32([1] * 100)
    cache.reserve(many, many)
    assert cache.device_status() == msa.MSA_ERR_BAD_INDEX
    cache.fork(i32([0] * 100), many)
    assert cache.device_status() == msa.MSA_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(tables(cache), was))
    cache.free(many)
    assert cache.device_status() == 0


def test_fork_without_pages_changes_nothing():
    """More partly filled last pages than free pages."""
    from block_sparse_long_index_gb300 import PagedCache, msa
    n_pages, page = 8, 16
    pools = [torch.arange(n_pages * page * 4, dtype=torch.int32, device="cuda").view(n_pages, page, 4)]
    cache = PagedCache.empty(6, 4, n_pages, page, pools)
    cache.reserve(i32([0, 1]), i32([40, 33]))  # 3 + 3 pages, both last ones partly filled: 2 free
    was = tables(cache)
    for src, dst in (([0, 1, 0], [2, 3, 4]), ([1, 1, 1, 1], [5, 4, 3, 2])):
        cache.fork(i32(src), i32(dst))
        assert cache.device_status() == msa.MSA_ERR_NO_PAGES
        assert all(torch.equal(a, b) for a, b in zip(tables(cache), was))
    cache.fork(i32([0, 1]), i32([2, 3]))  # as many as there are
    assert cache.device_status() == 0 and cache.ctx_len.tolist() == [40, 33, 40, 33, 0, 0]
    assert torch.equal(pools[0][cache.page_table[2, 2]], was[3][was[0][0, 2]])
    was = tables(cache)
    cache.fork(i32([1]), i32([4]))
    assert cache.device_status() == msa.MSA_ERR_NO_PAGES
    assert all(torch.equal(a, b) for a, b in zip(tables(cache), was))


def test_free_clears_the_entries():
    """What a freed sequence held reads -1; entries past it and other sequences stay as they were."""
    from block_sparse_long_index_gb300 import PagedCache
    cache = PagedCache.empty(4, 6, 16, 16)
    cache.reserve(i32([0, 1, 2]), i32([70, 16, 48]))
    cache.page_table[0, 5] = 77  # past the length: neither read nor written
    keep = cache.page_table[1:2].clone()
    cache.free(i32([0, 3, 2]))  # (3 is empty)
    assert cache.device_status() == 0 and cache.ctx_len.tolist() == [0, 16, 0, 0]
    assert cache.page_table[0].tolist() == [-1] * 5 + [77] and cache.page_table[2].tolist() == [-1] * 6
    assert torch.equal(cache.page_table[1:2], keep) and int(cache.refs.sum()) == 1


# ---------------------------------------------------------------- two calls at once
def test_two_prefills_at_once():
    """Two plans, made before, on two streams: out and lse of both, rows of no sequence, and both statuses."""
    from block_sparse_long_index_gb300 import MsaDensePrefill
    cases = [([900, 50], 8, 1, 128), ([20, 700], 8, 8, 64)]
    ins = [make(*c, pad=5, seed=i) for i, c in enumerate(cases)]
    plans = [MsaDensePrefill(q.shape[0], q.shape[1], k.shape[1], q.shape[2], 2) for q, k, _, _ in ins]
    want = [[t.clone() for t in p(*x, 0.1)] for p, x in zip(plans, ins)]
    streams = [torch.cuda.Stream() for _ in plans]
    for _ in range(4):
        for p in plans:
            p.out.fill_(7.0)
            p.lse.fill_(7.0)
        torch.cuda.synchronize()
        for p, x, s in zip(plans, ins, streams):
            p(*x, 0.1, stream=s)
        torch.cuda.synchronize()
        for p, (o, l), (lens, _, _, _) in zip(plans, want, cases):
            n = sum(lens)
            assert p.device_status() == 0
            assert torch.equal(p.out[:n], o[:n]) and torch.equal(p.lse[:, :n], l[:, :n])
            assert bool((p.out[n:] == 7.0).all()) and bool((p.lse[:, n:] == 7.0).all())


def test_stores_and_loads_at_once():
    """Other sequences of one pool on two streams (the pool's error word is the only thing that they share)."""
    from block_sparse_long_index_gb300 import Kv4Pool
    page, H, d = 16, 2, 128
    for n in (5, 900):  # calls whose status one CTA writes, and calls that clear it before
        pages = -(-n // page)
        pool = Kv4Pool.empty(2 * pages, page, H, d)
        ids = torch.randperm(2 * pages, device="cuda").to(torch.int32).view(2, 1, pages).contiguous()
        cu, pos = i32([0, n]), i32([0])
        x, streams = [rnd(n, H, d) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
        got = [[torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            pool.store(x[i], x[1 - i], cu, pos, ids[i], stream=s)
            pool.load(n, cu, pos, ids[i], *got[i], stream=s)
        torch.cuda.synchronize()
        assert pool.device_status() == 0
        assert torch.equal(got[0][0], got[1][1]) and torch.equal(got[0][1], got[1][0])
        k, v = pool.load(n, cu, pos, ids[0])
        assert torch.equal(k, got[0][0]) and torch.equal(v, got[0][1]) and bool((k != 0).any())


# ---------------------------------------------------------------- captured calls
def test_captured_prefill_with_a_plan_of_its_own():
    """More sequences than a warp has lanes: the planning kernel and its dependent in one graph, other offsets a replay."""
    from block_sparse_long_index_gb300 import MsaDensePrefill
    S, d = 40, 64
    lens = [(11 * i) % 37 for i in range(S)]
    q, k, v, cu = make(lens, 4, 2, d, pad=50)
    N = q.shape[0]
    plan = MsaDensePrefill(N, 4, 2, d, S)
    plan(q, k, v, cu, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(q, k, v, cu, 0.1)
    for step in (5, 17, 0):
        lens = [(step * i) % 23 for i in range(S)] if step else [0] * (S - 1) + [N]
        n = sum(lens)
        cu.copy_(torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32))
        plan.out.fill_(7.0)
        plan.lse.fill_(7.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        ref.check_attention(plan.out[:n], plan.lse[:, :n].T, *ref.dense_prefill(q[:n], k[:n], v[:n], lens, 0.1), d, max(lens))
        assert bool((plan.out[n:] == 7.0).all()) and bool((plan.lse[:, n:] == 7.0).all())


def test_captured_page_cycle():
    """Reserve, fork, free and compact in one graph, replayed on the state that the replay before left."""
    from test_gpu_pages import Both
    b = Both(6, 8, 60, 16)
    grow, to, src, dst, gone = i32([0, 1]), i32([70, 40]), i32([0, 1, 0]), i32([2, 3, 4]), i32([0, 3])
    b.gpu.reserve(grow, to)
    b.gpu.free(grow)
    b.gpu.fork(i32([5]), i32([4]))  # (an empty one: kernels loaded before the capture)
    b.gpu.compact()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.gpu.reserve(grow, to)
        b.gpu.fork(src, dst)
        b.gpu.free(gone)
        page_map, n_live = b.gpu.compact()
    for rest in ([1, 2, 4], [4, 2, 1], [2, 1, 4]):
        graph.replay()
        torch.cuda.synchronize()
        assert b.gpu.device_status() == 0
        b.ref.reserve([0, 1], [70, 40])
        b.ref.fork([0, 1, 0], [2, 3, 4])
        b.ref.free([0, 3])
        want, n = b.ref.compact()
        assert page_map.tolist() == want and n_live.tolist() == [n]
        b.check()
        b.gpu.free(i32(rest))
        b.ref.free(rest)
        b.check()


# ---------------------------------------------------------------- status
def test_status_is_that_of_the_last_call():
    """A call with bad data sets it, the next call without clears it, whichever kernel of a call writes it."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4, MsaDensePrefill, PagedCache, msa
    bad, no_pages = msa.MSA_ERR_BAD_INDEX, msa.MSA_ERR_NO_PAGES
    for S in (1, 40):  # planned by the CTAs, by a kernel
        plan, x = MsaDensePrefill(80, 2, 1, 64, S), [rnd(80, h, 64) for h in (2, 1, 1)]
        good, wrong = i32([2 * i for i in range(S + 1)]), i32([1] * (S + 1))
        for cu, want in ((wrong, bad), (good, 0), (wrong, bad)):
            plan(*x, cu)
            assert plan.device_status() == want
    for n in (5, 300):
        pool, x = Kv4Pool.empty(30, 16, 1, 64), rnd(n, 1, 64)
        good, wrong = i32([list(range(20))]), i32([[99] * 20])
        for table, want in ((wrong, bad), (good, 0), (wrong, bad), (good, 0)):
            pool.store(x, x, i32([0, n]), i32([0]), table)
            assert pool.device_status() == want
            pool.load(n, i32([0, n]), i32([0]), table)
            assert pool.device_status() == want
    run = MsaDecodeKv4(pool, 2, 20, 2, d_I=64, Bk=64, k=2)
    q, qi, ki, table = rnd(2, 2, 64), rnd(2, 1, 64), rnd(30, 16, 64), i32([list(range(20)), list(range(10, 30))])
    for ctx, want in (([-1, 5], bad), ([30, 300], 0), ([20, 321], bad), ([1, 320], 0)):
        run.dense(q, table, i32(ctx))
        assert run.device_status() == want
        run(q, qi, ki, table, i32(ctx))
        assert run.device_status() == want
        run.dense(q, table, i32([7, 7]))
        assert run.device_status() == 0
    cache = PagedCache.empty(3, 4, 4, 16)
    for seqs, lens, want in (([3], [1], bad), ([0], [20], 0), ([1, 2], [33, 1], no_pages), ([1], [10], 0)):
        cache.reserve(i32(seqs), i32(lens))
        assert cache.device_status() == want
    for src, dst, want in (([0], [1], bad), ([0], [2], 0)):
        cache.fork(i32(src), i32(dst))
        assert cache.device_status() == want
    for seqs, want in (([7], bad), ([2], 0)):
        cache.free(i32(seqs))
        assert cache.device_status() == want
    cache.page_table[0, 0] = 77
    cache.compact()
    assert cache.device_status() == bad
    cache.free(i32([]))
    assert cache.device_status() == 0
