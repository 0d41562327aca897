"""Rotary positions and rows into the paged caches on the GPU, against rotations in 64 bits and against the calls that do the
same in two steps."""
import math

import numpy as np
import pytest
import torch

import draft_ref as ref
from serving_ref import BF16_HALF
from test_gpu_kv4 import cu_of, i32, rows_of, table_of

pytestmark = pytest.mark.gpu


def freqs_of(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def rows(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check_turned(y, x, positions, freqs, interleaved=False, amplitude=1.0, inverse=False):
    want = ref.turn(x.double(), positions, freqs, interleaved, amplitude, inverse)
    tol = ref.turn_error(x.double(), freqs, positions, interleaved, amplitude)
    if y.dtype == torch.bfloat16:
        tol = tol * (1 + BF16_HALF) + BF16_HALF * want.abs() + 2.0 ** -134  # (half the smallest subnormal)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), "worst %.3f of the tolerance" % float((err / tol.clamp_min(1e-300)).max())
    n = 2 * len(freqs)
    assert torch.equal(y[..., n:], x[..., n:])


# ---------------------------------------------------------------- rows by themselves
ROPE = [
    # N, H, d, rot, interleaved, first position, amplitude
    (1, 1, 32, 16, False, 0, 1.0),
    (3, 5, 64, 64, False, 4095, 1.0),
    (7, 3, 64, 32, True, 1, 1.0),
    (50, 32, 128, 128, False, 1 << 20, 1.0),
    (33, 9, 128, 64, True, 999_983, 1.0),
    (17, 1, 256, 256, False, (1 << 31) - 17, 1.0),
    (5, 2, 256, 48, True, -3, 1.25),
    (1300, 2, 128, 96, False, 131000, 0.875),  # more tokens a CTA than one
    (10007, 3, 32, 32, True, 5, 1.0),
]


@pytest.mark.parametrize("N,H,d,rot,inter,first,amp", ROPE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_turned(N, H, d, rot, inter, first, amp, dtype):
    from block_sparse_long_index_gb300 import Rope
    x = rows(N, H, d, dtype=dtype, seed=N)
    pos = [first + i for i in range(N)]
    rope = Rope.from_frequencies(freqs_of(rot), interleaved=inter, amplitude=amp)
    for inverse in (False, True):
        y = rope(x, i32(pos), inverse=inverse)
        check_turned(y, x, pos, freqs_of(rot), inter, amp, inverse)


def test_positions_in_any_order_rows_apart_and_in_place():
    from block_sparse_long_index_gb300 import Rope
    N, H, d = 40, 4, 64
    wide = rows(N, 3 * H * d, seed=1)
    x = wide[:, H * d:2 * H * d].unflatten(1, (H, d))  # the middle third of a projection
    pos = np.random.default_rng(0).integers(-5, 1 << 20, N).tolist()
    rope = Rope(d, base=500000.0, scaling="linear", factor=8.0)
    freqs = [f / 8 for f in freqs_of(d, 500000.0)]
    y = rope(x, i32(pos))
    check_turned(y, x, pos, freqs)
    before = wide.clone()
    assert rope(x, i32(pos), out=x) is x and torch.equal(x, y)
    wide_now = wide.clone()
    wide_now[:, H * d:2 * H * d] = before[:, H * d:2 * H * d]
    assert torch.equal(wide_now, before)  # nothing beside the rows is written
    assert rope(rows(0, H, d), i32([])).shape == (0, H, d)


def test_gradient_is_the_transpose():
    """<rope(x), g> = <x, rope^T(g)>, and the gradient of a loss against differences of it (both in 64 bits of fp32 rows)."""
    from block_sparse_long_index_gb300 import Rope
    N, H, d = 12, 3, 64
    x, g = rows(N, H, d, dtype=torch.float32, seed=2), rows(N, H, d, dtype=torch.float32, seed=3)
    pos = list(range(100_000, 100_000 + N))
    freqs = freqs_of(32)
    rope = Rope.from_frequencies(freqs, amplitude=1.5)
    dx = rope(g, i32(pos), inverse=True)
    lhs = (rope(x, i32(pos)).double() * g.double()).sum()
    rhs = (x.double() * dx.double()).sum()
    tol = (ref.turn_error(x.double(), freqs, pos, amplitude=1.5) * g.abs()).sum() + (ref.turn_error(g.double(), freqs, pos, amplitude=1.5) * x.abs()).sum()
    assert abs(float(lhs - rhs)) <= float(tol)
    loss = lambda z: (ref.turn(z, pos, freqs, amplitude=1.5) * g.double()).sum()  # noqa: E731
    for at in ((0, 0, 0), (5, 1, 17), (11, 2, 40), (3, 0, 31)):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[at] = 0.5  # the loss is linear: any step gives its slope
        slope = loss(x.double() + e) - loss(x.double() - e)
        err = ref.turn_error(g.double(), freqs, pos, amplitude=1.5)[at]
        assert abs(float(slope - dx[at].double())) <= float(err) + 1e-10


def test_rows_that_are_not_finite_stay_by_themselves():
    from block_sparse_long_index_gb300 import Rope
    x = rows(6, 2, 64, seed=4)
    clean = x.clone()
    x[2, 1, 5], x[4, 0, 63] = math.nan, math.inf  # 5 turns with 5 + 16; 63 does not turn
    rope = Rope(32)
    y, want = rope(x, i32(range(6))), rope(clean, i32(range(6)))
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[2, 1, 5] = bad[2, 1, 21] = bad[4, 0, 63] = True
    assert torch.equal(y[~bad], want[~bad]) and bool(y[2, 1, [5, 21]].isnan().all()) and float(y[4, 0, 63]) == math.inf


def test_rope_refusals():
    from block_sparse_long_index_gb300 import Rope, msa
    rope, x, pos = Rope(64), rows(4, 2, 64), i32(range(4))
    for bad in (lambda: rope(x.half(), pos), lambda: rope(x.cpu(), pos), lambda: rope(x[0], pos), lambda: rope(x, pos.long()),
                lambda: rope(x, pos[:3]), lambda: rope(x.transpose(1, 2), pos), lambda: rope(x, pos, out=x[:3]),
                lambda: rope(x, pos, out=x.float()), lambda: rope(x.expand(4, 2, 64)[:1].expand(4, 2, 64), pos)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(msa.MsaError):  # rows that begin off a multiple of 16 bytes
        rope(rows(4, 2 * 64 + 4)[:, 4:].unflatten(1, (2, 64)), pos)
    with pytest.raises(msa.MsaError):  # more channels than the rows have
        Rope(128)(x, pos)


# ---------------------------------------------------------------- rows into the caches
APPEND = [
    # lens, pos0, H_q, H_kv, d, rot, interleaved, d_I, idx, page
    ([1], [0], 1, 1, 64, 64, False, 0, "bf16", 16),
    ([1, 1, 1, 1], [0, 15, 16, 40], 8, 2, 128, 128, False, 128, "bf16", 16),
    ([5, 0, 33], [14, 3, 0], 3, 3, 64, 32, True, 32, "bf16", 32),
    ([130, 7], [0, 121], 0, 8, 128, 64, False, 64, "fp8", 64),
    ([50], [77], 10, 5, 128, 16, True, 128, "fp8", 48),
    ([700, 1, 3000], [5, 0, 100], 6, 3, 64, 48, False, 64, "bf16", 80),  # several tokens a CTA
]


def state(lens, pos0, H_kv, d, page, seed=0):
    counts = [-(-(p + n) // page) for n, p in zip(lens, pos0)]
    n_pages = sum(counts) + 3
    return table_of(counts, max(max(counts), 1) + 1, n_pages, seed), n_pages


@pytest.mark.parametrize("lens,pos0,H_q,H_kv,d,rot,inter,d_I,idx,page", APPEND)
@pytest.mark.parametrize("own_positions", [False, True])
def test_append(lens, pos0, H_q, H_kv, d, rot, inter, d_I, idx, page, own_positions):
    """The bf16 pool holds the turned rows; the 4-bit pool the codes, bit for bit, that store makes of them."""
    from block_sparse_long_index_gb300 import Kv4Pool, KvPool, Rope, msa
    N = sum(lens)
    table, n_pages = state(lens, pos0, H_kv, d, page)
    wide = rows(N, (H_q + 2 * H_kv) * d, seed=N)  # queries, keys and values side by side, as a projection leaves them
    q = wide[:, :H_q * d].unflatten(1, (H_q, d)) if H_q else None
    k, v = (wide[:, (H_q + i * H_kv) * d:(H_q + (i + 1) * H_kv) * d].unflatten(1, (H_kv, d)) for i in (0, 1))
    k_idx, q_idx = (rows(N, d_I, seed=7), rows(N, H_kv, d_I, seed=8)) if d_I else (None, None)
    rope, freqs = Rope.from_frequencies(freqs_of(rot), interleaved=inter), freqs_of(rot)
    rot_i = min(rot, d_I)
    idx_rope = Rope.from_frequencies(freqs_of(rot_i, 500.0)) if d_I else None
    places = [p + i for n, p in zip(lens, pos0) for i in range(n)]
    pos = [3 * p - 50 for p in places] if own_positions else places
    where = torch.tensor(rows_of(lens, pos0, table, page), device="cuda")
    turned = rope(k, i32(pos))  # (checked against 64 bits by itself; append's is to be equal)
    check_turned(turned, k, pos, freqs, inter)
    f8 = idx == "fp8"
    pools, outs = [KvPool.empty(n_pages, page, H_kv, d), Kv4Pool.empty(n_pages, page, H_kv, d)], []
    other = Kv4Pool.empty(n_pages, page, H_kv, d)
    for pool in pools:
        for t in pool.tensors():
            t.fill_(7)
        k_idx_pool = torch.full((n_pages, page, d_I), 7, dtype=torch.uint8 if f8 else torch.bfloat16, device="cuda") if d_I else None
        got = pool.append(k, v, cu_of(lens), i32(pos0), table, rope=rope, positions=i32(pos) if own_positions else None, q=q,
                          k_idx=k_idx, k_idx_pool=k_idx_pool, q_idx=q_idx, idx_rope=idx_rope, idx_scale=0.5)
        assert pool.device_status() == 0
        outs.append((*got, k_idx_pool))
    for a, b in zip(*outs):
        assert (a is None and b is None) or torch.equal(a, b)
    bf = pools[0]
    untouched = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    untouched[where] = False
    assert torch.equal(bf.k.flatten(0, 1)[where], turned) and torch.equal(bf.v.flatten(0, 1)[where], v)
    assert bool((bf.k.flatten(0, 1)[untouched] == 7).all()) and bool((bf.v.flatten(0, 1)[untouched] == 7).all())
    for t in other.tensors():
        t.fill_(7)
    other.store(turned, v.contiguous(), cu_of(lens), i32(pos0), table)
    assert all(torch.equal(a, b) for a, b in zip(other.tensors(), pools[1].tensors()))
    got_q, got_qi, held = outs[0]
    if H_q:
        assert torch.equal(got_q, rope(q, i32(pos)))
    if d_I:
        ti, tq = idx_rope(k_idx[:, None], i32(pos))[:, 0].contiguous(), idx_rope(q_idx, i32(pos))
        check_turned(ti[:, None], k_idx[:, None], pos, freqs_of(rot_i, 500.0))
        if f8:
            codes = [torch.empty(t.shape, dtype=torch.uint8, device="cuda") for t in (ti, tq)]
            for t, c in zip((ti, tq), codes):
                msa.msa_quantize_e4m3(t, t.numel(), 0.5, c)
            ti, tq = codes
        assert torch.equal(held.flatten(0, 1)[where], ti) and torch.equal(got_qi, tq)
        assert bool((held.flatten(0, 1)[untouched] == 7).all())


def test_append_without_rotation_and_parts():
    from block_sparse_long_index_gb300 import Kv4Pool, KvPool
    lens, pos0, page = [9, 4], [0, 30], 16
    table, n_pages = state(lens, pos0, 2, 64, page)
    k, v, ki = rows(13, 2, 64, seed=1), rows(13, 2, 64, seed=2), rows(13, 64, seed=3)
    where = torch.tensor(rows_of(lens, pos0, table, page), device="cuda")
    pool, held = KvPool.empty(n_pages, page, 2, 64), torch.zeros((n_pages, page, 64), dtype=torch.bfloat16, device="cuda")
    assert pool.append(k, v, cu_of(lens), i32(pos0), table, k_idx=ki, k_idx_pool=held) == (None, None)
    assert torch.equal(pool.k.flatten(0, 1)[where], k) and torch.equal(held.flatten(0, 1)[where], ki)
    a, b = Kv4Pool.empty(n_pages, page, 2, 64), Kv4Pool.empty(n_pages, page, 2, 64)
    a.append(k, v, cu_of(lens), i32(pos0), table)
    b.store(k, v, cu_of(lens), i32(pos0), table)
    assert all(torch.equal(x, y) for x, y in zip(a.tensors(), b.tensors()))


@pytest.mark.parametrize("many", [False, True])
def test_append_passes_over_rows_without_a_place(many):
    """Rows of no sequence and rows with bad pages or positions: nothing of theirs is written, the others are as always."""
    from block_sparse_long_index_gb300 import KvPool, Rope, msa
    page, n_pages = 16, 40
    lens = [300, 20, 6] if many else [3, 20, 6]  # (few rows: one CTA reports)
    N = sum(lens) + 5
    table, _ = state(lens, [0, 0, 0], 1, 64, page)
    table = torch.cat([table, torch.full_like(table[:, :3], -1)], 1).contiguous()
    n_pages = int(table.max()) + 1
    table[1, 1] = n_pages  # tokens 16 .. of the second
    pos0 = [0, 0, table.shape[1] * page - 4]  # the third runs past its table, and its pages are -1
    k, v, q = rows(N, 1, 64, seed=1), rows(N, 1, 64, seed=2), rows(N, 2, 64, seed=3)
    pool, rope = KvPool.empty(n_pages, page, 1, 64), Rope(64)
    out = torch.full_like(q, 7)
    pool.append(k, v, cu_of(lens), i32(pos0), table, rope=rope, q=q, q_out=out)
    assert pool.device_status() == msa.MSA_ERR_BAD_INDEX
    good = lens[0] + 16
    want = rope(q, i32(list(range(lens[0])) + list(range(20)) + [0] * (N - lens[0] - 20)))
    assert torch.equal(out[:good], want[:good]) and bool((out[good:] == 7).all())
    where = torch.tensor(rows_of([lens[0], 16], [0, 0], table, page), device="cuda")
    assert torch.equal(pool.v.flatten(0, 1)[where], v[:good])
    left = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    left[where] = False
    assert not bool(pool.v.flatten(0, 1)[left].any()) and not bool(pool.k.flatten(0, 1)[left].any())
    pool.append(k[:1], v[:1], cu_of([1]), i32([0]), table[:1])
    assert pool.device_status() == 0  # the next call clears it


def test_append_into_a_pool_past_32_bit_offsets():
    from block_sparse_long_index_gb300 import KvPool, Rope
    H_kv, d, page = 8, 128, 128
    n_pages = (1 << 31) // (page * H_kv * d) + 40  # past 2^31 elements, 2^32 bytes
    pool = KvPool(torch.empty((n_pages, page, H_kv, d), dtype=torch.bfloat16, device="cuda"),
                  torch.empty((n_pages, page, H_kv, d), dtype=torch.bfloat16, device="cuda"))
    table = i32([[n_pages - 1, 0, n_pages - 2]])
    k, v = rows(300, H_kv, d, seed=1), rows(300, H_kv, d, seed=2)
    rope = Rope(d)
    pool.append(k, v, cu_of([300]), i32([40]), table, rope=rope)
    assert pool.device_status() == 0
    got = [torch.cat([t[n_pages - 1, 40:], t[0], t[n_pages - 2, :84]]) for t in pool.tensors()]
    assert torch.equal(got[0], rope(k, i32(range(40, 340)))) and torch.equal(got[1], v)


def test_append_on_another_stream_and_captured():
    from block_sparse_long_index_gb300 import Kv4Pool, Rope
    lens, page = [1] * 20, 32
    table = table_of([2] * 20, 2, 41)
    pos0 = i32(range(20))
    k, v, q = rows(20, 4, 128, seed=1), rows(20, 4, 128, seed=2), rows(20, 8, 128, seed=3)
    rope = Rope(64)
    want = Kv4Pool.empty(41, page, 4, 128)
    want_q, _ = want.append(k, v, cu_of(lens), pos0, table, rope=rope, q=q)
    pool, cu, s = Kv4Pool.empty(41, page, 4, 128), cu_of(lens), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got_q, _ = pool.append(k, v, cu, pos0, table, rope=rope, q=q, stream=s)
    s.synchronize()
    assert torch.equal(got_q, want_q) and all(torch.equal(a, b) for a, b in zip(pool.tensors(), want.tensors()))
    pool = Kv4Pool.empty(41, page, 4, 128)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.append(k, v, cu, pos0, table, rope=rope, q=q, q_out=out)
    k.copy_(rows(20, 4, 128, seed=9))
    pos0.add_(11)
    g.replay()
    torch.cuda.synchronize()
    want = Kv4Pool.empty(41, page, 4, 128)
    want_q, _ = want.append(k, v, cu, pos0, table, rope=rope, q=q)
    assert torch.equal(out, want_q) and all(torch.equal(a, b) for a, b in zip(pool.tensors(), want.tensors()))


def test_append_refusals():
    from block_sparse_long_index_gb300 import KvPool, Rope
    pool, k = KvPool.empty(4, 16, 2, 64), rows(3, 2, 64)
    cu, pos, table, ki = cu_of([3]), i32([0]), i32([[0, 1]]), rows(3, 32)
    held = torch.zeros((4, 16, 32), dtype=torch.bfloat16, device="cuda")
    good = dict(k=k, v=k, cu_seqlens=cu, pos0=pos, page_table=table)
    pool.append(**good)
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(v=k.cpu()), dict(cu_seqlens=cu.long()), dict(pos0=i32([0, 1])),
                dict(page_table=table[0]), dict(positions=i32([1])), dict(q=rows(3, 2, 128)), dict(q=rows(2, 2, 64)),
                dict(k_idx=ki), dict(k_idx_pool=held), dict(k_idx=ki, k_idx_pool=held[:3]), dict(q=k, q_out=k.float()),
                dict(k_idx=ki, k_idx_pool=held, q_idx=rows(3, 2, 64)), dict(k=k.transpose(1, 2)), dict(rope=Rope(32, device="cpu"))):
        with pytest.raises(ValueError):
            pool.append(**{**good, **bad})
