"""Keys and values that are not finite: a NaN that is attended reaches the outputs of its heads, one that is not
attended reaches none; a key whose score is -inf weighs nothing, and a row without another is like an empty one."""
import math

import pytest
import torch

import serving_ref as ref
from test_gpu_dense_prefill import make, run
from test_gpu_kv4 import dense_ref, i32, random_pool, table_of

pytestmark = pytest.mark.gpu

SHAPES = [
    # ctx, k, token with the NaN, H_q, H_kv, d, Bk, page; sequence 1 stays clean
    ([50, 40], 4, 20, 8, 2, 64, 64, 16),       # one valid slot of several
    ([200, 190], 1, 199, 16, 2, 128, 128, 64),  # one slot
    ([300, 500], 8, 299, 16, 2, 128, 64, 32),   # the local block of several
    ([300, 500], 8, 70, 8, 8, 64, 64, 16),      # another chosen block
    ([700, 900], 8, 3, 4, 4, 128, 128, 48),
]


def step_inputs(ctx, H_q, H_kv, d, page, index):
    from block_sparse_long_index_gb300 import msa
    counts = [-(-c // page) for c in ctx]
    n_pages, B = sum(counts) + 2, len(ctx)
    pool, table = random_pool(n_pages, page, H_kv, d), table_of(counts, max(counts), n_pages)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, qi, ki = rnd(B, H_q, d), rnd(B, H_kv, 64), rnd(n_pages, page, 64)
    if index == "fp8":
        codes = [torch.empty(t.shape, dtype=torch.uint8, device="cuda") for t in (qi, ki)]
        for t, c in zip((qi, ki), codes):
            msa.msa_quantize_e4m3(t, t.numel(), 16.0, c)
        qi, ki = codes
    return pool, table, q, qi, ki


def step(pool, table, q, qi, ki, ctx, Bk, k):
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    run = MsaDecodeKv4(pool, len(ctx), table.shape[1], q.shape[1], d_I=64, Bk=Bk, k=k)
    run.out.fill_(7.0)
    run.lse.fill_(7.0)
    got = [t.clone() for t in run(q, qi, ki, table, i32(ctx), 0.1)]
    assert run.device_status() == 0
    return got


def place(table, b, token, page):
    return int(table[b, token // page]), token % page


@pytest.mark.parametrize("index", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,k,token,H_q,H_kv,d,Bk,page", SHAPES)
def test_step_over_nan_groups(ctx, k, token, H_q, H_kv, d, Bk, page, index):
    pool, table, q, qi, ki = step_inputs(ctx, H_q, H_kv, d, page, index)
    out, lse, blk = step(pool, table, q, qi, ki, ctx, Bk, k)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    gs, g = H_q // H_kv, H_kv - 1
    hit = slice(g * gs, g * gs + gs)
    at = place(table, 0, token, page)
    # a group of K: every score of the token is NaN, so everything of its heads is
    keep = pool.k_scales[at[0], at[1], g, 2].clone()
    pool.k_scales[at[0], at[1], g, 2] = 255
    o, l, b = step(pool, table, q, qi, ki, ctx, Bk, k)
    assert token // Bk in blk[0, g].tolist() and torch.equal(b, blk)
    assert bool(torch.isnan(o[0, hit]).all()) and bool(torch.isnan(l[0, hit]).all())
    o[0, hit], l[0, hit] = out[0, hit], lse[0, hit]
    assert torch.equal(o, out) and torch.equal(l, lse)
    pool.k_scales[at[0], at[1], g, 2] = keep
    # a group of V: its channels alone
    pool.v_scales[at[0], at[1], g, 1] = 255
    o, l, _ = step(pool, table, q, qi, ki, ctx, Bk, k)
    c = slice(d // 4, d // 2)
    assert bool(torch.isnan(o[0, hit, c]).all()) and torch.equal(l, lse)
    o[0, hit, c] = out[0, hit, c]
    assert torch.equal(o, out)


def test_step_leaves_out_nan_groups_that_it_does_not_attend():
    """Blocks that were not chosen, and tokens past the length."""
    ctx, Bk, k, page = [1000, 130], 64, 3, 16
    pool, table, q, qi, ki = step_inputs(ctx, 8, 2, 64, page, "bf16")
    out, lse, blk = step(pool, table, q, qi, ki, ctx, Bk, k)
    for b, n in enumerate(ctx):
        for t in range(table.shape[1] * page):
            if table[b, t // page] < 0:
                continue
            for g in range(2):
                if t >= n or t // Bk not in blk[b, g].tolist():
                    p, r = place(table, b, t, page)
                    pool.k_scales[p, r, g] = 255
                    pool.v_scales[p, r, g] = 255
    o, l, b = step(pool, table, q, qi, ki, ctx, Bk, k)
    assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(b, blk)


def test_step_from_stored_infinities():
    """What store makes of an infinity in K is a NaN of the step, whole context or chosen blocks."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4
    N, H_kv, d, page = 90, 2, 128, 16
    pool = Kv4Pool.empty(6, page, H_kv, d)
    k, v = (torch.randn(N, H_kv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    k[33, 1, 5] = math.inf
    table, cu, pos = i32([[3, 0, 5, 1, 4, 2]]), i32([0, N]), i32([0])
    pool.store(k, v, cu, pos, table)
    q, qi = torch.randn(1, 4, d, device="cuda").to(torch.bfloat16), torch.randn(1, H_kv, 64, device="cuda").to(torch.bfloat16)
    ki = torch.randn(6, page, 64, device="cuda").to(torch.bfloat16)
    run = MsaDecodeKv4(pool, 1, 6, 4, d_I=64, Bk=64, k=2)
    for o, l in (run.dense(q, table, i32([N]), 0.1), run(q, qi, ki, table, i32([N]), 0.1)[:2]):
        assert bool(torch.isnan(o[0, 2:]).all()) and bool(torch.isnan(l[0, 2:]).all())
        assert bool(torch.isfinite(o[0, :2]).all()) and bool(torch.isfinite(l[0, :2]).all())


@pytest.mark.parametrize("ctx", [[40, 30], [200, 90]])
def test_bf16_steps_over_nan(ctx):
    """The same of the steps over bf16 caches, contiguous and paged."""
    from block_sparse_long_index_gb300 import msa
    B, H_q, H_kv, d, N = 2, 8, 2, 64, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, qi, ki, k, v = rnd(B, H_q, d), rnd(B, H_kv, 64), rnd(B, N, 64), rnd(B, N, H_kv, d), rnd(B, N, H_kv, d)
    shape = msa.shape(N, H_q, H_kv, d, 64, 64, 4)
    ws = torch.empty(msa.msa_decode_workspace(B, shape), dtype=torch.uint8, device="cuda")
    table = i32([list(range(16)), list(range(16, 32))])

    def both():
        got = []
        for paged in (False, True):
            o, l = torch.empty_like(q), torch.empty(B, H_q, device="cuda")
            if paged:
                msa.msa_decode_paged(q, qi, ki, k, v, table, 16, 32, 16, i32(ctx), B, shape, 0.1, o, l, None, ws)
            else:
                msa.msa_decode(q, qi, ki, k, v, i32(ctx), B, shape, 0.1, o, l, None, ws)
            assert msa.msa_check_device_error(ws) == 0
            got.append((o, l))
        assert torch.equal(got[0][0].isnan(), got[1][0].isnan())
        return got

    clean = both()
    k[0, 11, 1, 7] = math.nan
    for (o, l), (co, cl) in zip(both(), clean):
        assert bool(torch.isnan(o[0, 4:]).all()) and bool(torch.isnan(l[0, 4:]).all())
        o[0, 4:], l[0, 4:] = co[0, 4:], cl[0, 4:]
        assert torch.equal(o, co) and torch.equal(l, cl)


# ---------------------------------------------------------------- scores of -inf
def seen_attention(q, k, v, lens, dead, scale):
    """ref.dense_prefill with the tokens marked in `dead` [N] taken out of every row's keys."""
    N, H_q, d = q.shape
    gs = H_q // k.shape[1]
    k = torch.where(dead[:, None, None], 0, k.double())
    out, A = (torch.zeros(N, H_q, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, S = torch.full((N, H_q), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(N, H_q, dtype=torch.float64, device="cuda")
    a = 0
    for n in lens:
        r = slice(a, a + n)
        mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril() & ~dead[None, r]
        some = mask.any(1)
        for h in range(H_q if bool(some.any()) else 0):
            kk, vv, qq = k[r, h // gs], v[r, h // gs].double(), q[r, h].double()
            x = (qq @ kk.T * scale).masked_fill(~mask, -math.inf)[some]
            ls = torch.logsumexp(x, 1)
            p = torch.exp(x - ls[:, None])
            rows = torch.arange(a, a + n, device="cuda")[some]
            out[rows, h], lse[rows, h], A[rows, h] = p @ vv, ls, p @ vv.abs()
            S[rows, h] = (qq.abs() @ kk.abs().T).masked_fill(~mask, 0).amax(1)[some] * scale
        a += n
    return out, lse, A, S


@pytest.mark.parametrize("H_q,H_kv,d", [(8, 1, 128), (2, 2, 64), (4, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("lens,dead", [
    ([1], [(0, 1)]),                       # one row
    ([1, 40, 1], [(0, 1), (1, 6), (41, 42)]),
    ([400], [(0, 256)]),                   # the first key tiles, and whole items where a tile holds few positions
    ([300], [(128, 256)]),                 # a tile in the middle
    ([140, 270], [(0, 140), (140, 145), (270, 410)]),
])
def test_prefill_scores_of_minus_infinity(lens, dead, H_q, H_kv, d):
    q, k, v, cu = make(lens, H_q, H_kv, d)
    q[:, :, 3] = 1.0
    marked = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
    for a, b in dead:
        marked[a:b] = True
    k[marked, :, 3] = -math.inf
    plan, out, lse = run(q, k, v, cu, 0.1)
    assert plan.device_status() == 0
    o, l, A, S = seen_attention(q, k, v, lens, marked, 0.1)
    none = l[:, 0] == -math.inf
    assert bool(none.any()) == (dead[0][0] == 0)
    assert bool((out[none] == 0).all()) and bool((lse.T[none] == -math.inf).all())
    ref.check_attention(out, lse.T, o, l, A, S, d, max(lens))


@pytest.mark.parametrize("d,H_kv", [(64, 1), (128, 2), (64, 8)])
@pytest.mark.parametrize("ctx", [[1, 5, 0], [16, 300, 31], [9000, 40, 7000]])
def test_dense_decode_scores_of_minus_infinity(ctx, H_kv, d):
    """Rows that one CTA holds and rows that several share.  (The query's infinity meets codes of one sign.)"""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    page = 16
    counts = [-(-c // page) for c in ctx]
    pool, table = random_pool(sum(counts) + 1, page, H_kv, d), table_of(counts, max(counts), sum(counts) + 1)
    pool.k_codes[..., 0] |= 0xF  # channel 0: the largest code
    q = torch.randn(3, 4 * H_kv, d, device="cuda").to(torch.bfloat16)
    plan = MsaDecodeKv4(pool, 3, table.shape[1], 4 * H_kv)
    want = [t[:, ::2] for t in dense_ref(pool, q, table, ctx, 0.1)]
    q[:, 1::2, 0] = -math.inf
    plan.out.fill_(7.0)
    plan.lse.fill_(7.0)
    out, lse = plan.dense(q, table, i32(ctx), 0.1)
    assert plan.device_status() == 0
    assert bool((out[:, 1::2] == 0).all()) and bool((lse[:, 1::2] == -math.inf).all())
    # (not the bits of a call without them: a warp moves the maxima that its 8 heads' sums refer to together, and any
    # reference within 2^8 gives the same sums up to the roundings that the tolerance counts)
    ref.check_attention(out[:, ::2], lse[:, ::2], *want, d, max(ctx))


@pytest.mark.parametrize("index", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,k,H_q,H_kv,d,Bk,page", [([1, 50], 3, 8, 2, 64, 64, 16), ([200, 700], 1, 16, 2, 128, 128, 64),
                                                      ([300, 900], 8, 8, 8, 128, 64, 32)])
def test_step_scores_of_minus_infinity(ctx, k, H_q, H_kv, d, Bk, page, index):
    pool, table, q, qi, ki = step_inputs(ctx, H_q, H_kv, d, page, index)
    pool.k_codes[..., 0] |= 0xF  # channel 0: the largest code
    want, want_lse, blk = step(pool, table, q, qi, ki, ctx, Bk, k)
    q[1, ::2, 0] = -math.inf
    out, lse, b = step(pool, table, q, qi, ki, ctx, Bk, k)
    assert bool((out[1, ::2] == 0).all()) and bool((lse[1, ::2] == -math.inf).all())
    want[1, ::2], want_lse[1, ::2] = 0, -math.inf
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(b, blk)  # (a head has its own maximum here)


def test_bf16_step_blocks_of_minus_infinity():
    """A chosen block whose scores are all -inf adds nothing to the others."""
    from block_sparse_long_index_gb300 import msa
    B, H_q, H_kv, d, N = 2, 8, 2, 128, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, qi, ki, k, v = rnd(B, H_q, d), rnd(B, H_kv, 64), rnd(B, N, 64), rnd(B, N, H_kv, d), rnd(B, N, H_kv, d)
    q[:, :, 3] = 1.0
    k[0, 64:128, :, 3] = -math.inf
    k[0, 200:, :, 3] = -math.inf  # a part of a block
    k[1, :, 1, 3] = -math.inf     # every key of a head
    shape = msa.shape(N, H_q, H_kv, d, 64, 64, 4)
    ws = torch.empty(msa.msa_decode_workspace(B, shape), dtype=torch.uint8, device="cuda")
    table = i32([list(range(16)), list(range(16, 32))])
    ctx = i32([256, 130])
    for paged in (False, True):
        o, l = torch.full_like(q, 7.0), torch.full((B, H_q), 7.0, device="cuda")
        if paged:
            msa.msa_decode_paged(q, qi, ki, k, v, table, 16, 32, 16, ctx, B, shape, 0.1, o, l, None, ws)
        else:
            msa.msa_decode(q, qi, ki, k, v, ctx, B, shape, 0.1, o, l, None, ws)
        assert msa.msa_check_device_error(ws) == 0
        assert bool((o[1, 4:] == 0).all()) and bool((l[1, 4:] == -math.inf).all())
        rows = torch.cat([torch.arange(64), torch.arange(128, 200)]).cuda()
        for b, h, at in ((0, 0, rows), (0, 1, rows), (1, 0, torch.arange(130).cuda())):
            hs = slice(4 * h, 4 * h + 4)
            r = ref.attend(q[b, hs].double(), k[b, at, h].double(), v[b, at, h].double(), 0.1)
            ref.check_attention(o[b, hs], l[b, hs], *r, d, 256)


@pytest.mark.parametrize("token", [0, 5000, 8999])
@pytest.mark.parametrize("H_kv,d", [(1, 128), (2, 64), (8, 128), (9, 64)])
def test_dense_decode_over_nan_groups(token, H_kv, d):
    """In a row that many CTAs share: everything of its heads for a group of K, its channels for a group of V."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    ctx, page = [9000, 40], 16
    counts = [-(-c // page) for c in ctx]
    pool, table = random_pool(sum(counts), page, H_kv, d), table_of(counts, max(counts), sum(counts))
    q = torch.randn(2, 4 * H_kv, d, device="cuda").to(torch.bfloat16)
    plan = MsaDecodeKv4(pool, 2, table.shape[1], 4 * H_kv)
    want = dense_ref(pool, q, table, ctx, 0.1)
    p, r = place(table, 0, token, page)
    hit, c = slice(4 * H_kv - 4, 4 * H_kv), slice(d // 4, d // 2)
    for scales in (pool.k_scales, pool.v_scales):
        keep = scales[p, r, H_kv - 1, 1].clone()
        scales[p, r, H_kv - 1, 1] = 255
        out, lse = [t.clone() for t in plan.dense(q, table, i32(ctx), 0.1)]
        assert plan.device_status() == 0
        scales[p, r, H_kv - 1, 1] = keep
        at = (0, hit) if scales is pool.k_scales else (0, hit, c)
        assert bool(torch.isnan(out[at]).all())
        out[at] = want[0][at].to(torch.bfloat16)
        if scales is pool.k_scales:
            assert bool(torch.isnan(lse[0, hit]).all())
            lse[0, hit] = want[1][0, hit].float()
        ref.check_attention(out, lse, *want, d, max(ctx))
