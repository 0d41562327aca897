"""The 4-bit paged cache on the GPU: rows in and out against the format's definition, dense decode and the MSA
step over it against 64-bit attention on the values that the codes stand for."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


def table_of(counts, max_pages, n_pages, seed=0):
    """Shuffled page ids for `counts` pages a sequence; the rest of the table is -1."""
    ids = np.random.default_rng(seed).permutation(n_pages)
    t = np.full((len(counts), max_pages), -1, np.int32)
    at = 0
    for s, c in enumerate(counts):
        t[s, :c] = ids[at:at + c]
        at += c
    return torch.from_numpy(t).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32([sum(lens[:i]) for i in range(len(lens) + 1)])


# ---------------------------------------------------------------- store and load
STORE = [
    # lens, pos0, H_kv, d, page
    ([1], [0], 1, 64, 16),
    ([1, 1, 1, 1], [0, 15, 16, 40], 2, 128, 16),
    ([5, 0, 33], [14, 3, 0], 3, 64, 32),
    ([130, 7], [0, 121], 8, 128, 64),
    ([50], [77], 5, 128, 48),
]


def rows_of(lens, pos0, table, page):
    t = table.cpu().numpy()
    return [int(t[s, p // page]) * page + p % page for s, (n, a) in enumerate(zip(lens, pos0)) for p in range(a, a + n)]


def tricky(N, H, d, seed):
    """Rows with ties, zeros, tiny and huge values, subnormals and lone outliers beside normal ones."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((N, H, d)).astype(np.float32)
    x[r.random(x.shape) < 0.1] = 0
    kind = r.integers(0, 8, (N, H, 4))
    g = x.reshape(N, H, 4, -1)
    g[kind == 1] *= 1e-7
    g[kind == 2] *= 1e5
    g[kind == 3] = 0
    k4 = kind == 4  # exact ties: halves of the scale that the group's largest value gives
    g[k4] = (r.integers(-14, 15, g[k4].shape) * 0.5 * 1.125 * 2.0 ** -3)
    g[kind == 5] *= 1e-39
    k6 = np.argwhere(kind == 6)
    for a, b, c in k6:
        g[a, b, c, r.integers(g.shape[-1])] = 300.0
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("lens,pos0,H,d,page", STORE)
def test_store_and_load(lens, pos0, H, d, page):
    from block_sparse_long_index_gb300 import Kv4Pool
    counts = [-(-(a + n) // page) for n, a in zip(lens, pos0)]
    n_pages, N = sum(counts) + 3, sum(lens)
    table = table_of(counts, max(counts) + 1, n_pages)
    pool = Kv4Pool.empty(n_pages, page, H, d)
    for t in pool.tensors():
        t.fill_(0x5A)
    k, v = tricky(N + 4, H, d, 1), tricky(N + 4, H, d, 2)  # the last 4 rows belong to no sequence
    pool.store(k.cuda(), v.cuda(), cu_of(lens), i32(pos0), table)
    assert pool.device_status() == 0
    rows = rows_of(lens, pos0, table, page)
    untouched = np.setdiff1d(np.arange(n_pages * page), rows)
    got = {}
    for x, codes, scales, name in ((k, pool.k_codes, pool.k_scales, "k"), (v, pool.v_codes, pool.v_scales, "v")):
        c, s = codes.cpu().numpy().reshape(-1, H, d // 2), scales.cpu().numpy().reshape(-1, H, 4)
        want_c, want_s = ref.quantize(x[:N].double().numpy())
        assert np.array_equal(s[rows], want_s), name
        assert np.array_equal(c[rows], ref.pack(want_c)), name
        assert (c[untouched] == 0x5A).all() and (s[untouched] == 0x5A).all(), name
        got[name] = ref.values(want_c, want_s)
    ko = torch.full((N + 4, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pool.load(N + 4, cu_of(lens), i32(pos0), table, ko, vo)
    assert pool.device_status() == 0
    for o, name in ((ko, "k"), (vo, "v")):
        assert np.array_equal(o[:N].double().cpu().numpy(), got[name]), name  # exact in bf16
        assert bool((o[N:] == 7.0).all())


def test_every_code_and_scale_expands_exactly():
    from block_sparse_long_index_gb300 import Kv4Pool
    page, H, d = 256, 1, 64
    pool = Kv4Pool.empty(1, page, H, d)
    codes = np.tile(np.arange(16), (page, 4))[:, None, :]  # all codes in every group of 16
    scales = np.repeat(np.arange(256), 4).reshape(page, 1, 4)  # token t: scale byte t in its four groups
    pool.k_codes.copy_(torch.from_numpy(ref.pack(codes))[None])
    pool.k_scales.copy_(torch.from_numpy(scales.astype(np.uint8))[None])
    k, _ = pool.load(page, cu_of([page]), i32([0]), i32([[0]]))
    want = ref.values(codes, scales)
    assert np.array_equal(k.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[255]).all() and np.isfinite(want[:255]).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_groups(bad):
    from block_sparse_long_index_gb300 import Kv4Pool
    pool = Kv4Pool.empty(1, 16, 2, 128)
    k = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    k[1, 0, 70] = bad
    pool.store(k, k, cu_of([3]), i32([0]), i32([[0]]))
    out, _ = pool.load(3, cu_of([3]), i32([0]), i32([[0]]))
    nan = torch.isnan(out)
    assert bool(nan[1, 0, 64:96].all()) and int(nan.sum()) == 32


def test_store_bad_places():
    from block_sparse_long_index_gb300 import Kv4Pool, msa
    pool = Kv4Pool.empty(4, 16, 1, 64)
    x = torch.ones(6, 1, 64, device="cuda", dtype=torch.bfloat16)
    cases = [(cu_of([6]), i32([28]), i32([[0, 1]])),      # the last two rows outside the table
             (cu_of([3, 3]), i32([0, -1]), i32([[0], [1]])),  # a negative position
             (cu_of([3, 3]), i32([0, 0]), i32([[0], [4]])),   # page ids outside the pool
             (cu_of([3, 3]), i32([0, 0]), i32([[0], [-1]]))]
    for cu, pos, table in cases:
        for t in pool.tensors():
            t.zero_()
        pool.store(x, x, cu, pos, table)
        assert pool.device_status() == msa.MSA_ERR_BAD_INDEX
        written = int((pool.k_scales.flatten(0, 1)[:, 0, 0] != 0).sum())
        assert written == (4 if cu.numel() == 2 else 3)
        k, _ = pool.load(6, cu, pos, table)
        assert pool.device_status() == msa.MSA_ERR_BAD_INDEX
        assert int((k[:, 0, 0] != 0).sum()) == written and bool(torch.isfinite(k).all())


# ---------------------------------------------------------------- decode
def random_pool(n_pages, page, H, d, seed=0):
    from block_sparse_long_index_gb300 import Kv4Pool
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pool = Kv4Pool.empty(n_pages, page, H, d)
    for t in (pool.k_codes, pool.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (pool.k_scales, pool.v_scales):
        t.copy_(torch.randint(120, 160, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return pool


def pool_values(pool):
    return [torch.from_numpy(ref.values(ref.unpack(c.cpu().numpy()), s.cpu().numpy().astype(np.int64))).cuda().flatten(0, 1)
            for c, s in ((pool.k_codes, pool.k_scales), (pool.v_codes, pool.v_scales))]


def dense_ref(pool, q, table, ctx, scale, tokens=None):
    """Whole-context attention in 64 bits; tokens[b][g] restricts a group's tokens."""
    K, V = pool_values(pool)
    B, H_q, d = q.shape
    gs, parts = H_q // pool.H_kv, []
    t = table.cpu().numpy()
    for b in range(B):
        for g in range(pool.H_kv):
            tok = range(ctx[b]) if tokens is None else tokens[b][g]
            rows = torch.tensor([int(t[b, j // pool.page_size]) * pool.page_size + j % pool.page_size for j in tok],
                                dtype=torch.long, device="cuda")
            parts.append(ref.attend(q[b, g * gs:(g + 1) * gs].double(), K[rows, g], V[rows, g], scale))
    return [torch.stack([p[i] for p in parts]).reshape((B, H_q) + tuple(parts[0][i].shape[1:])) for i in range(4)]


DECODE = [
    # ctx, H_q, H_kv, d, page
    ([1], 1, 1, 64, 16),
    ([0], 8, 1, 128, 16),
    ([0, 5, 0, 17], 4, 2, 64, 16),
    ([16, 15, 17, 1], 8, 8, 128, 32),
    ([130, 1000, 64, 3], 16, 2, 128, 48),
    ([2500], 8, 2, 64, 64),
    ([700, 0, 31, 1200, 1], 24, 3, 128, 128),
    ([333, 90], 48, 6, 64, 16),
    ([5000, 20], 12, 12, 128, 128),
    ([1500], 8, 1, 128, 80),
    ([100] * 70, 16, 16, 64, 16),
]


@pytest.mark.parametrize("ctx,H_q,H_kv,d,page", DECODE)
def test_dense_decode(ctx, H_q, H_kv, d, page):
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    counts = [-(-c // page) for c in ctx]
    n_pages = sum(counts) + 2
    pool, table = random_pool(n_pages, page, H_kv, d), table_of(counts, max(max(counts), 1), n_pages)
    q = torch.randn(len(ctx), H_q, d, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, len(ctx), table.shape[1], H_q)
    run.out.fill_(7.0)
    scale = 1 / math.sqrt(d)
    out, lse = run.dense(q, table, i32(ctx), scale)
    assert run.device_status() == 0
    o, l, A, S = dense_ref(pool, q, table, ctx, scale)
    ref.check_attention(out, lse, o, l, A, S, d, max(ctx + [1]))


def test_dense_decode_large_scores_and_repeat():
    """Maxima that rise along the cache, and equal bits from equal calls."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    ctx, page, H_kv, d = [2200, 900], 64, 2, 128
    counts = [-(-c // page) for c in ctx]
    pool, table = random_pool(sum(counts), page, H_kv, d), table_of(counts, max(counts), sum(counts))
    order = torch.empty(sum(counts), dtype=torch.long)
    order[table[table >= 0].cpu().long()] = torch.arange(sum(counts))
    pool.k_scales.copy_((100 + order.cuda()[:, None, None, None]).clamp(max=165).expand_as(pool.k_scales))
    q = torch.randn(2, 16, d, device="cuda").mul(3).to(torch.bfloat16)
    run = MsaDecodeKv4(pool, 2, table.shape[1], 16)
    out, lse = run.dense(q, table, i32(ctx), 0.2)
    o, l, A, S = dense_ref(pool, q, table, ctx, 0.2)
    ref.check_attention(out, lse, o, l, A, S, d, max(ctx))
    first = out.clone()
    for _ in range(3):
        assert torch.equal(run.dense(q, table, i32(ctx), 0.2)[0], first)


def test_dense_decode_stale_rows():
    """Tokens past the length hold NaN scales (a page's earlier owner): they reach no output."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    ctx, page, H_kv, d = [21, 40, 7], 16, 2, 64
    pool, table = random_pool(9, page, H_kv, d), table_of([3, 3, 3], 3, 9)
    t = table.cpu().numpy()
    for b, n in enumerate(ctx):
        for j in range(n, 48):
            for s in (pool.k_scales, pool.v_scales):
                s[int(t[b, j // page]), j % page] = 255
    q = torch.randn(3, 4, d, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, 3, 3, 4)
    out, lse = run.dense(q, table, i32(ctx), 0.1)
    assert run.device_status() == 0
    ref.check_attention(out, lse, *dense_ref(pool, q, table, ctx, 0.1), d, 40)


def test_dense_decode_errors():
    from block_sparse_long_index_gb300 import MsaDecodeKv4, msa
    pool = random_pool(6, 16, 2, 64)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, 3, 2, 4)
    out, lse = run.dense(q, i32([[0, 1], [2, 3], [4, 5]]), i32([20, -1, 33]), 0.1)
    assert run.device_status() == msa.MSA_ERR_BAD_INDEX
    assert bool((out[1:] == 0).all()) and bool((lse[1:] == -math.inf).all())
    ref.check_attention(out[:1], lse[:1], *dense_ref(pool, q[:1], i32([[0, 1]]), [20], 0.1), 64, 20)
    run.dense(q, i32([[0, 9], [2, 3], [-1, 5]]), i32([20, 5, 3]), 0.1)
    assert run.device_status() == msa.MSA_ERR_BAD_INDEX
    assert bool(torch.isfinite(out).all())  # page 0 read in place of a bad one


def test_dense_decode_graph_and_streams():
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    page, H_kv, d = 32, 4, 128
    pool, table = random_pool(40, page, H_kv, d), table_of([20, 20], 20, 40)
    q = torch.randn(2, 8, d, device="cuda").to(torch.bfloat16)
    ctx = i32([600, 33])
    a, b = MsaDecodeKv4(pool, 2, 20, 8), MsaDecodeKv4(pool, 2, 20, 8)
    want = a.dense(q, table, ctx, 0.1)[0].clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.dense(q, table, ctx, 0.1, stream=s1)
        b.dense(q, table, ctx, 0.1, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and torch.equal(b.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.dense(q, table, ctx, 0.1)
    for n in ([601, 34], [0, 640], [17, 1]):  # the lengths are read on the device
        ctx.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert a.device_status() == 0
        ref.check_attention(a.out, a.lse, *dense_ref(pool, q, table, n, 0.1), d, max(n))


STEP = [
    # ctx, H_q, H_kv, d, d_I, Bk, k, page, fp8
    ([1], 1, 1, 64, 32, 64, 1, 16, False),
    ([700, 64, 65], 8, 2, 64, 64, 64, 4, 16, False),
    ([1500, 129, 3], 16, 2, 128, 128, 128, 3, 64, False),
    ([900, 2000], 32, 8, 128, 64, 64, 16, 128, False),
    ([1111], 3, 3, 128, 128, 128, 20, 80, False),
    ([700, 64, 65], 8, 2, 128, 64, 64, 4, 16, True),
    ([1500, 129, 3], 16, 2, 64, 128, 128, 3, 64, True),
]


@pytest.mark.parametrize("ctx,H_q,H_kv,d,d_I,Bk,k,page,fp8", STEP)
def test_msa_step(ctx, H_q, H_kv, d, d_I, Bk, k, page, fp8):
    """Sets equal to the bf16 step's on the same index keys, attention on the step's own sets in 64 bits."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4, msa
    counts = [-(-c // page) for c in ctx]
    n_pages, B = sum(counts) + 2, len(ctx)
    pool, table = random_pool(n_pages, page, H_kv, d), table_of(counts, max(counts), n_pages)
    q = torch.randn(B, H_q, d, device="cuda").to(torch.bfloat16)
    qi, ki = torch.randn(B, H_kv, d_I, device="cuda").to(torch.bfloat16), torch.randn(n_pages, page, d_I, device="cuda").to(torch.bfloat16)
    if fp8:
        codes = [torch.empty(t.shape, dtype=torch.uint8, device="cuda") for t in (qi, ki)]
        for t, c in zip((qi, ki), codes):
            msa.msa_quantize_e4m3(t, t.numel(), 16.0, c)
        qi, ki = codes
    run = MsaDecodeKv4(pool, B, table.shape[1], H_q, d_I=d_I, Bk=Bk, k=k)
    out, lse, blk = run(q, qi, ki, table, i32(ctx), 0.1)
    assert run.device_status() == 0
    # the bf16 step over the values of the same codes
    kb, vb = [t.to(torch.bfloat16).reshape(n_pages, page, H_kv, d) for t in pool_values(pool)]
    o2, l2, b2 = torch.empty_like(out), torch.empty_like(lse), torch.empty_like(blk)
    ws = torch.empty(msa.msa_decode_workspace(B, run.shape), dtype=torch.uint8, device="cuda")
    call = msa.msa_decode_paged_fp8 if fp8 else msa.msa_decode_paged
    call(q, qi, ki, kb, vb, table, table.shape[1], n_pages, page, i32(ctx), B, run.shape, 0.1, o2, l2, b2, ws)
    torch.cuda.synchronize()
    assert torch.equal(blk, b2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)  # the same arithmetic on the same values
    tokens = [[[j for b in sorted(set(r)) if b >= 0 for j in range(b * Bk, min(b * Bk + Bk, n))] for r in rows]
              for rows, n in zip(blk.cpu().tolist(), ctx)]
    o, l, A, S = dense_ref(pool, q, table, ctx, 0.1, tokens)
    # the partials of k blocks are merged once more in fp32
    ref.check_attention(out, lse, o, l, A, S, d, k * Bk)


def test_msa_step_every_block_is_dense():
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    ctx, page = [500, 130], 64
    pool, table = random_pool(12, page, 2, 128), table_of([8, 3], 8, 12)
    q, qi = torch.randn(2, 16, 128, device="cuda").to(torch.bfloat16), torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)
    ki = torch.randn(12, page, 64, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, 2, 8, 16, d_I=64, Bk=64, k=8)
    a = [t.clone() for t in run(q, qi, ki, table, i32(ctx), 0.1)[:2]]
    b = run.dense(q, table, i32(ctx), 0.1)
    assert float((a[0].float() - b[0].float()).norm() / b[0].float().norm()) < 2 * ref.BF16_HALF
    assert float((a[1] - b[1]).abs().max()) < 1e-5


def test_dense_decode_every_code_and_scale():
    """One token a sequence: its output is V itself, so each (code, scale) pair is seen to be exact, the largest
    and the smallest ones, and NaN scales, among them."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    for d in (64, 128):
        pool = random_pool(256, 16, 1, d)
        codes = np.tile(np.arange(16), d // 16)
        pool.v_codes[:, 0] = torch.from_numpy(ref.pack(codes[None])).cuda()
        pool.v_scales[:, 0] = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None, None]
        q = torch.randn(256, 8, d, device="cuda").to(torch.bfloat16)
        run = MsaDecodeKv4(pool, 256, 1, 8)
        out, _ = run.dense(q, torch.arange(256, dtype=torch.int32, device="cuda")[:, None], i32([1] * 256), 0.1)
        want = ref.values(np.broadcast_to(codes, (256, d)), np.repeat(np.arange(256), 4).reshape(256, 4))
        got = out.double().cpu().numpy()
        assert all(np.array_equal(got[:, h], want, equal_nan=True) for h in range(8))
