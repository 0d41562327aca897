"""The serving operators where a size chooses another path: many sequences or rows, every head block, pools and
batches past 32-bit offsets, and the calls of a decode step captured together."""
import math
import random

import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_dense_prefill import make, run
from test_gpu_kv4 import cu_of, dense_ref, i32, random_pool, rows_of, table_of
from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- dense prefill
@pytest.mark.parametrize("lens,H_q,H_kv,d", [
    ([(7 * i) % 23 for i in range(33)], 8, 2, 128),       # more sequences than a warp has lanes
    ([1] * 400, 4, 4, 64),
    ([i % 3 * 130 for i in range(40)], 8, 1, 128),
    ([3000, 0, 700, 1300], 32, 8, 64),                    # many items: planned by a kernel of their own
    ([2500], 64, 64, 128),
    ([1, 2049, 0, 2047], 24, 24, 64),
])
def test_prefill_planned_apart(lens, H_q, H_kv, d):
    q, k, v, cu = make(lens, H_q, H_kv, d, pad=3)
    n, scale = sum(lens), 1 / math.sqrt(d)
    plan, out, lse = run(q, k, v, cu, scale)
    assert plan.device_status() == 0
    ref.check_attention(out[:n], lse[:, :n].T, *ref.dense_prefill(q[:n], k[:n], v[:n], lens, scale), d, max(lens))
    assert bool((out[n:] == 7.0).all()) and bool((lse[:, n:] == 7.0).all())


def test_prefill_past_32_bit_offsets():
    """More than 2^32 bytes and 2^31 elements of q: each sequence equals the call on it alone."""
    from block_sparse_long_index_gb300 import MsaDensePrefill
    S, n, H_q, H_kv, d = 2100, 128, 64, 8, 128
    N = S * n
    assert N * H_q * d > 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q, k, v = (torch.randn(N, h, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (H_q, H_kv, H_kv))
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    plan = MsaDensePrefill(N, H_q, H_kv, d, S)
    out, lse = plan(q, k, v, cu)
    assert plan.device_status() == 0
    one = MsaDensePrefill(n, H_q, H_kv, d, 1)
    for s in (0, 1, 1023, 2047, 2048, S - 1):  # row 2048 x 128 starts past 2^31 elements
        r = slice(s * n, (s + 1) * n)
        o, l = one(q[r], k[r], v[r], cu[:2])
        ref.check_attention(o, l.T, *ref.dense_prefill(q[r], k[r], v[r], [n], 1 / math.sqrt(d)), d, n)
        assert torch.equal(out[r], o) and torch.equal(lse[:, r], l), s


# ---------------------------------------------------------------- 4-bit rows
def quantize(x):
    """ref.quantize for finite values, without its loop: the first scale that reaches the largest value."""
    g = x.reshape(*x.shape[:-1], 4, -1)
    sv = ref.scale_values()
    s = np.minimum(np.searchsorted(7 * sv, np.abs(g).max(-1), side="left"), 254)
    codes = 8 + np.clip(np.rint(g / sv[s][..., None]), -7, 7).astype(np.int64)
    return codes.reshape(x.shape), s


@pytest.mark.parametrize("H,d,N,page", [(1, 64, 80000, 16), (2, 128, 41111, 64), (3, 64, 30001, 48), (5, 128, 9000, 16),
                                        (8, 128, 12000, 128), (64, 64, 2500, 32), (33, 128, 2600, 16)])
def test_store_and_load_many_rows(H, d, N, page):
    from block_sparse_long_index_gb300 import Kv4Pool
    lens, pos0 = [N // 3, 0, 1, N - N // 3 - 1], [5, 0, 31, 0]
    counts = [-(-(a + n) // page) for n, a in zip(lens, pos0)]
    n_pages = sum(counts) + 2
    table = table_of(counts, max(counts), n_pages)
    pool = Kv4Pool.empty(n_pages, page, H, d)
    for t in pool.tensors():
        t.fill_(0x5A)
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    k, v = (torch.randn(N + 9, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    v *= torch.exp2(torch.randint(-24, 12, (N + 9, H, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    pool.store(k, v, cu_of(lens), i32(pos0), table)
    assert pool.device_status() == 0
    rows = rows_of(lens, pos0, table, page)
    untouched = np.setdiff1d(np.arange(n_pages * page), rows)
    ko = torch.full((N + 9, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pool.load(N + 9, cu_of(lens), i32(pos0), table, ko, vo)
    assert pool.device_status() == 0
    for x, codes, scales, o in ((k, pool.k_codes, pool.k_scales, ko), (v, pool.v_codes, pool.v_scales, vo)):
        c, s = codes.cpu().numpy().reshape(-1, H, d // 2), scales.cpu().numpy().reshape(-1, H, 4)
        want_c, want_s = quantize(x[:N].double().cpu().numpy())
        few = ref.quantize(x[:3].double().cpu().numpy())
        assert np.array_equal(few[0], want_c[:3]) and np.array_equal(few[1], want_s[:3])
        assert np.array_equal(s[rows], want_s) and np.array_equal(c[rows], ref.pack(want_c))
        assert (c[untouched] == 0x5A).all() and (s[untouched] == 0x5A).all()
        assert np.array_equal(o[:N].double().cpu().numpy(), ref.values(want_c, want_s))
        assert bool((o[N:] == 7.0).all())


# ---------------------------------------------------------------- dense decode
@pytest.mark.parametrize("ctx,H_q,H_kv,d,page", [
    ([300, 41], 5, 5, 64, 16),                     # heads that do not fill the last head block
    ([300, 41, 2000], 28, 7, 128, 32),
    ([177, 1, 90], 9, 9, 128, 16),
    ([250, 33], 64, 64, 128, 16),
    ([250, 33], 128, 64, 64, 48),
    ([700], 8, 1, 64, 16),
    ([(37 * i) % 90 for i in range(300)], 4, 2, 64, 16),   # more rows than CTAs
    ([(53 * i) % 70 for i in range(700)], 8, 8, 128, 32),
    ([1] * 1000, 4, 1, 128, 16),
    ([3] * 40 + [4000] + [2] * 40, 8, 4, 128, 64),
])
def test_decode_shapes(ctx, H_q, H_kv, d, page):
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    counts = [-(-c // page) for c in ctx]
    n_pages = sum(counts) + 2
    pool, table = random_pool(n_pages, page, H_kv, d), table_of(counts, max(counts), n_pages)
    q = torch.randn(len(ctx), H_q, d, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, len(ctx), table.shape[1], H_q)
    run.out.fill_(7.0)
    out, lse = run.dense(q, table, i32(ctx), 0.11)
    assert run.device_status() == 0
    ref.check_attention(out, lse, *dense_ref(pool, q, table, ctx, 0.11), d, max(ctx))


def test_pool_past_32_bit_offsets():
    """Pages whose codes lie past 2^32 bytes hold, give and attend to the same bits as those of a small pool."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4, PagedCache
    page, H, d, d_I, n_big = 128, 8, 128, 64, 70000
    assert n_big * page * H * d // 2 > 1 << 32
    big, small = Kv4Pool.empty(n_big, page, H, d), Kv4Pool.empty(8, page, H, d)
    lens, pos0 = [300, 200], [0, 100]
    t_small = i32([[0, 5, 2], [7, 1, 3]])
    t_big = i32([[n_big - 1, 40000, 33000], [66000, n_big - 7, 2]])
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v, k0, v0 = rnd(500, H, d), rnd(500, H, d), rnd(100, H, d), rnd(100, H, d)
    ki_big = torch.empty(n_big, page, d_I, dtype=torch.bfloat16, device="cuda")
    ki_small = rnd(8, page, d_I)
    ki_big[t_big.flatten().long()] = ki_small[t_small.flatten().long()]
    q, qi = rnd(2, 64, d), rnd(2, H, d_I)
    got = []
    for pool, t, ki in ((small, t_small, ki_small), (big, t_big, ki_big)):
        pool.store(k0, v0, cu_of([0, 100]), i32([0, 0]), t)
        pool.store(k, v, cu_of(lens), i32(pos0), t)
        kv = pool.load(500, cu_of(lens), i32(pos0), t)
        run = MsaDecodeKv4(pool, 2, 3, 64, d_I=d_I, Bk=128, k=2)
        o = [x.clone() for x in run.dense(q, t, i32([300, 300]), 0.1)]
        s = run(q, qi, ki, t, i32([300, 300]), 0.1)
        assert pool.device_status() == 0 and run.device_status() == 0
        got.append(list(kv) + o + [x.clone() for x in s])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ref.check_attention(got[0][2], got[0][3], *dense_ref(small, q, t_small, [300, 300], 0.1), d, 300)
    # a fork copies a partial last page, compaction moves the high ones down
    refs = torch.zeros(n_big, dtype=torch.int32, device="cuda")
    refs[t_big.flatten().long()] = 1
    table = torch.cat([t_big, torch.full((2, 3), -1, dtype=torch.int32, device="cuda")])
    cache = PagedCache(table, i32([300, 300, 0, 0]), refs, page, big.tensors() + [ki_big])
    cache.fork(i32([0, 1]), i32([2, 3]))
    _, n = cache.compact()
    assert cache.device_status() == 0 and int(n) == 8 and int(cache.page_table.max()) == 7
    run = MsaDecodeKv4(big, 4, 3, 64, d_I=d_I, Bk=128, k=2)
    o, l = run.dense(q.repeat(2, 1, 1), cache.page_table, cache.ctx_len, 0.1)
    assert run.device_status() == 0
    # (equal inputs, but rows are split by the whole batch: the order of a row's sums may differ)
    ref.check_attention(o, l, *[x.repeat(2, *[1] * (x.dim() - 1)) for x in dense_ref(small, q, t_small, [300, 300], 0.1)], d, 300)
    k2, v2 = big.load(1000, cu_of([300, 200, 300, 200]), i32([0, 100, 0, 100]), cache.page_table)
    assert torch.equal(k2, got[0][0].repeat(2, 1, 1)) and torch.equal(v2, got[0][1].repeat(2, 1, 1))


# ---------------------------------------------------------------- pages
def test_pages_many_entries():
    """More entries a call and sequences than a CTA has threads."""
    r = random.Random(7)
    n_seqs, most, n_pages, page = 2600, 5, 9000, 16
    b = Both(n_seqs, most, n_pages, page)
    seqs = r.sample(range(n_seqs), 1300)
    lens = [r.randint(0, 4 * page) for _ in seqs]
    assert b.ref.reserve(seqs, lens)
    b.gpu.reserve(i32(seqs), i32(lens))
    b.check()
    empty = [s for s in range(n_seqs) if b.ref.ctx[s] == 0]
    dst = r.sample(empty, 1200)
    src = [r.choice(seqs) for _ in dst]
    assert b.ref.fork(src, dst)
    b.gpu.fork(i32(src), i32(dst))
    b.check()
    gone = [r.randrange(n_seqs) for _ in range(1500)]  # some of them twice, some empty
    b.ref.free(gone)
    b.gpu.free(i32(gone))
    b.check()
    page_map, n_live = b.ref.compact()
    m, n = b.gpu.compact()
    assert b.gpu.device_status() == 0 and m.tolist() == page_map and n.tolist() == [n_live]
    b.check()
    grow = [s for s in range(n_seqs) if b.ref.ctx[s]][:1100]
    to = [min(most * page, b.ref.ctx[s] + page) for s in grow]
    assert b.ref.reserve(grow, to)
    b.gpu.reserve(i32(grow), i32(to))
    assert b.gpu.device_status() == 0
    b.check()


# ---------------------------------------------------------------- a captured decode step
def test_captured_step():
    """Reserve, store, dense attention and the MSA step in one graph on a side stream: each replay adds a token and
    leaves the bits that the same calls leave one by one."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4, PagedCache
    H_q, H_kv, d, d_I, page, n_pages, B = 8, 2, 64, 32, 16, 40, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens = [70, 1, 32]
    k, v, ki = rnd(103, H_kv, d), rnd(103, H_kv, d), rnd(n_pages, page, d_I)
    kt, vt, q, qi = (torch.empty(B, h, w, dtype=torch.bfloat16, device="cuda")
                     for h, w in ((H_kv, d), (H_kv, d), (H_q, d), (H_kv, d_I)))

    class Arm:
        def __init__(self):
            self.pool = Kv4Pool.empty(n_pages, page, H_kv, d)
            for t in self.pool.tensors():
                t.zero_()
            self.cache = PagedCache.empty(B, 8, n_pages, page, self.pool.tensors())
            self.cache.reserve(i32([0, 1, 2]), i32(lens))
            self.pool.store(k, v, cu_of(lens), i32([0, 0, 0]), self.cache.page_table)
            self.run = MsaDecodeKv4(self.pool, B, 8, H_q, d_I=d_I, Bk=64, k=1)
            self.seqs, self.ones = i32([0, 1, 2]), i32([0, 1, 2, 3])
            self.before, self.after = i32(lens), i32(lens)
            self.dense = [torch.empty(B, H_q, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H_q, device="cuda")]

        def step(self):
            self.before.copy_(self.after)
            self.after.add_(1)
            self.cache.reserve(self.seqs, self.after)
            self.pool.store(kt, vt, self.ones, self.before, self.cache.page_table)
            for to, x in zip(self.dense, self.run.dense(q, self.cache.page_table, self.cache.ctx_len, 0.125)):
                to.copy_(x)
            self.run(q, qi, ki, self.cache.page_table, self.cache.ctx_len, 0.125)

        def state(self):
            return self.dense + [self.run.out, self.run.lse, self.cache.ctx_len, self.cache.refs] + self.pool.tensors()

    a, b = Arm(), Arm()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.step()
    for _ in range(20):
        for t in (kt, vt, q, qi):
            t.copy_(rnd(*t.shape))
        torch.cuda.synchronize()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        for x in (a, b):
            assert x.cache.device_status() == 0 and x.pool.device_status() == 0 and x.run.device_status() == 0
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    assert a.cache.ctx_len.tolist() == [n + 20 for n in lens]
    n = [x + 20 for x in lens]
    ref.check_attention(*a.dense, *dense_ref(a.pool, q, a.cache.page_table, n, 0.125), d, max(n))


@pytest.mark.parametrize("handle", [False, True])
def test_load_allocates_for_its_stream(handle):
    """Rows that a call on another stream makes do not take memory that the current stream still reads."""
    from block_sparse_long_index_gb300 import Kv4Pool
    N, H, d, page = 4096, 2, 128, 64
    pool = Kv4Pool.empty(N // page, page, H, d)
    table = i32([list(range(N // page))])
    x = torch.randn(N, H, d, device="cuda").to(torch.bfloat16)
    pool.store(x, x, cu_of([N]), i32([0]), table)
    want = pool.load(N, cu_of([N]), i32([0]), table)[0].clone()
    cu, pos, s = cu_of([N]), i32([0]), torch.cuda.Stream()
    old = torch.full((N, H, d), 3.0, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms on the current stream
    seen = old.clone()
    del old  # its block is free for the current stream, which still has to read it
    k, v = pool.load(N, cu, pos, table, stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    assert torch.equal(k, want) and torch.equal(v, want)
    assert bool((seen == 3.0).all())
