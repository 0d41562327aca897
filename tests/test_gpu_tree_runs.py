"""Attention of drafted trees where a CTA of the context kernel goes through several tiles, several sequences and several units:
two query tiles a unit over bf16 pages, and more K/V heads than fill the GPU in one round.  Against 64 bits."""
import math

import numpy as np
import pytest
import torch

import draft_ref as ref
import serving_ref as sref
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


def attend(q, k, v, ctx, parents, scale):
    """draft_ref.tree_attend with all nodes and heads of a K/V head at once."""
    T, H_q, d = q.shape
    H_kv, n = k.shape[1], k.shape[0]
    gs = H_q // H_kv
    sees = torch.zeros((T, n), dtype=torch.bool)
    sees[:, :ctx] = True
    for i, line in enumerate(ref.ancestors(parents)):
        sees[i, [ctx + j for j in line]] = True
    out, A = torch.zeros_like(q), torch.zeros_like(q)
    lse, S = (torch.zeros(T, H_q, dtype=torch.float64, device=q.device) for _ in range(2))
    hidden = ~sees.to(q.device)[:, None]
    for g in range(H_kv):
        qq, h = q[:, g * gs:(g + 1) * gs], slice(g * gs, (g + 1) * gs)
        x = torch.einsum("tgd,nd->tgn", qq, k[:, g]).mul_(scale).masked_fill_(hidden, -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, h, None])
        out[:, h], A[:, h] = p @ v[:, g], p @ v[:, g].abs()
        S[:, h] = torch.einsum("tgd,nd->tgn", qq.abs(), k[:, g].abs()).masked_fill_(hidden, 0.0).amax(-1) * scale
    return out, lse, A, S


def check(c, out, lse, only=None, tree_len=None):
    for b in range(c.B) if only is None else only:
        T = c.T if tree_len is None else tree_len[b]
        if T:
            k, v = c.values(b, c.ctx[b] + T)
            want, wl, A, S = attend(c.q[b, :T].double(), k, v, c.ctx[b], c.parents[b][:T], c.scale)
            sref.check_attention(out[b, :T].flatten(0, 1), lse[b, :T].flatten(), want.flatten(0, 1), wl.flatten(), A.flatten(0, 1),
                                 S.flatten(), c.d, c.ctx[b] + T)
        assert bool((out[b, T:] == 7).all()) and bool((lse[b, T:] == 7).all())


@pytest.mark.parametrize("T,H_q,H_kv,d,page", [
    (17, 16, 2, 128, 64),  # 136 rows: the second query tile has 8
    (64, 8, 2, 64, 128),   # 256
    (32, 64, 8, 128, 32),  # 256, longer runs
    (40, 16, 2, 128, 16),  # 320: the second row group has one query tile, half filled
    (64, 16, 2, 64, 48),   # 512
    (64, 32, 4, 128, 64),  # 512
])
def test_two_query_tiles_over_long_runs(T, H_q, H_kv, d, page):
    """One context that every CTA has several tiles of, with later maxima far above the first ones."""
    c = Case("bf16", [40000], T, H_q, H_kv, d, page, "random", seed=40 + T)
    pages, gs = c.table[0].long(), H_q // H_kv
    for i, t in enumerate(range(3000, 40000, 4099)):  # keys along the queries, each larger than the last
        c.pool.k[pages[t // page], t % page] = c.q[0, (7 * i) % T, ::gs] * (0.2 * i + 0.3)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    check(c, out, lse)
    again = tuple(t.clone() for t in (out, lse))
    out, lse = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("T,H_q,H_kv,d,page", [(17, 16, 2, 64, 16), (64, 16, 4, 128, 64), (64, 64, 8, 128, 128), (40, 8, 1, 128, 16)])
def test_two_query_tiles_over_many_sequences(T, H_q, H_kv, d, page):
    """Runs that go from sequence to sequence, empty ones and trees of other lengths between them."""
    r = np.random.default_rng(41)
    ctx = [int(x) for x in r.integers(0, 2600, 70)]
    ctx[3], ctx[4], ctx[20], ctx[21], ctx[69] = 0, 0, 128, 1, 9000
    tl = [T] * 70
    tl[7], tl[8], tl[30], tl[50] = 0, 1, T // 2, T - 1
    c = Case("bf16", ctx, T, H_q, H_kv, d, page, "random", seed=41 + T)
    out, lse = c.run(tree_len=tl)
    assert c.dec.device_status() == 0
    check(c, out, lse, only=[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 20, 21, 22, 30, 49, 50, 51, 67, 68, 69], tree_len=tl)


ROUNDS = [  # units (K/V heads, and groups of their rows) that leave many CTAs idle in one round
    (1, 28, 28, 64, 32), (2, 32, 32, 128, 64), (5, 40, 40, 64, 16), (3, 64, 64, 128, 16), (7, 14, 14, 128, 64), (4, 80, 20, 64, 48),
    (33, 32, 32, 64, 32), (64, 112, 14, 64, 64), (64, 64, 8, 128, 128), (40, 160, 20, 128, 32), (64, 512, 64, 64, 16),
]


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("T,H_q,H_kv,d,page", ROUNDS)
def test_rounds(kind, T, H_q, H_kv, d, page):
    big = H_q * T > 4096
    ctx = [300, 0, 129, 1500] if big else [0, 5000, 129, 1, 0, 2600, 128, 700, 12000]
    tl = [T] * len(ctx)
    tl[2] = max(T - 2, 1)
    c = Case(kind, ctx, T, H_q, H_kv, d, page, "random", seed=42 + T + H_kv)
    out, lse = c.run(tree_len=tl)
    assert c.dec.device_status() == 0
    check(c, out, lse, tree_len=tl)
    again = tuple(t.clone() for t in (out, lse))
    out, lse = c.run(tree_len=tl)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("B,T,H_q,H_kv,d", [(3, 1, 2, 2, 64), (60, 3, 24, 6, 128), (80, 9, 32, 8, 64), (150, 17, 16, 8, 128), (70, 5, 64, 8, 64)])
def test_joins_whose_warps_have_rows_or_none(kind, B, T, H_q, H_kv, d):
    """One, two and four tiles of 16 rows a CTA of the joining kernel, the last ones in part or not at all filled."""
    r = np.random.default_rng(43)
    ctx = [int(x) for x in r.integers(0, 60, B)]
    tl = [int(x) for x in r.integers(0, T + 1, B)]
    c = Case(kind, ctx, T, H_q, H_kv, d, 16, "random", seed=43 + T)
    out, lse = c.run(tree_len=tl)
    assert c.dec.device_status() == 0
    check(c, out, lse, tree_len=tl)
