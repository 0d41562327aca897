"""Attention of drafted trees over bf16 and 4-bit paged caches on the GPU, against 64-bit attention row by row."""
import math

import numpy as np
import pytest
import torch

import draft_ref as ref
import serving_ref as sref
from test_gpu_kv4 import i32, table_of
from test_gpu_rope import rows

pytestmark = pytest.mark.gpu


class Case:
    """A pool with random contents, tables, trees; `values` reads the cache of a sequence back in 64 bits."""

    def __init__(self, kind, ctx, T, H_q, H_kv, d, page, tree="random", seed=0, spare_cols=1):
        from block_sparse_long_index_gb300 import Kv4Pool, KvPool
        r = np.random.default_rng(seed)
        self.kind, self.ctx, self.T, self.H_q, self.H_kv, self.d, self.page = kind, ctx, T, H_q, H_kv, d, page
        self.B = len(ctx)
        counts = [-(-(n + T) // page) for n in ctx]
        self.n_pages = sum(counts) + 2
        self.table = table_of(counts, max(counts) + spare_cols, self.n_pages, seed)
        if kind == "bf16":
            self.pool = KvPool(rows(self.n_pages, page, H_kv, d, seed=seed), rows(self.n_pages, page, H_kv, d, seed=seed + 1))
        else:
            g = torch.Generator(device="cuda").manual_seed(seed)
            self.pool = Kv4Pool(*[torch.randint(lo, hi, (self.n_pages, page, H_kv, last), generator=g, device="cuda", dtype=torch.uint8)
                                  for lo, hi, last in ((0, 256, d // 2), (136, 156, 4)) * 2])
        self.q = rows(self.B, T, H_q, d, seed=seed + 2)
        self.parents = [ref.tree_of(r, T, tree) for _ in ctx]
        self.scale = 1.0 / math.sqrt(d)

    def values(self, b, n):
        """K and V of the first n tokens of sequence b."""
        t = self.table[b].long().cpu()
        at = torch.tensor([int(t[i // self.page]) * self.page + i % self.page for i in range(n)])
        if self.kind == "bf16":
            return [x.flatten(0, 1)[at.cuda()].double() for x in (self.pool.k, self.pool.v)]
        out = []
        for c, s in ((self.pool.k_codes, self.pool.k_scales), (self.pool.v_codes, self.pool.v_scales)):
            c, s = (x.flatten(0, 1)[at.cuda()].cpu().numpy() for x in (c, s))
            out.append(torch.tensor(sref.values(sref.unpack(c), s.astype(np.int64)), device="cuda"))
        return out

    def run(self, tree_len=None, **kw):
        from block_sparse_long_index_gb300 import MsaTreeDecode
        self.dec = MsaTreeDecode(self.pool, self.B, self.T, self.table.shape[1], self.H_q)
        self.dec.out.fill_(7)
        self.dec.lse.fill_(7)
        return self.dec(self.q, self.table, i32(self.ctx), i32(self.parents), None if tree_len is None else i32(tree_len),
                        self.scale, **kw)

    def check(self, out, lse, tree_len=None, only=None):
        for b in range(self.B) if only is None else only:
            T = self.T if tree_len is None else tree_len[b]
            if T == 0:
                assert bool((out[b] == 7).all()) and bool((lse[b] == 7).all())
                continue
            k, v = self.values(b, self.ctx[b] + T)
            want, wl, A, S = ref.tree_attend(self.q[b, :T].double(), k, v, self.ctx[b], self.parents[b][:T], self.scale)
            sref.check_attention(out[b, :T].flatten(0, 1), lse[b, :T].flatten(), want.flatten(0, 1), wl.flatten(), A.flatten(0, 1),
                                 S.flatten(), self.d, self.ctx[b] + T)
            assert bool((out[b, T:] == 7).all()) and bool((lse[b, T:] == 7).all())


TREES = [
    # ctx, T, H_q, H_kv, d, page, tree
    ([0], 1, 1, 1, 64, 16, "chain"),
    ([1], 1, 8, 1, 128, 16, "chain"),
    ([0, 5, 127, 128, 129], 3, 4, 2, 64, 16, "wide"),
    ([255, 256, 257, 0], 5, 6, 3, 128, 48, "random"),
    ([1500], 8, 8, 2, 64, 64, "chain"),
    ([700, 30, 2000], 16, 16, 2, 128, 128, "random"),  # 128 rows: one query tile filled
    ([600, 1], 17, 16, 2, 128, 80, "random"),  # 136 rows: two query tiles
    ([333, 1000], 64, 4, 1, 64, 32, "random"),  # 256 rows
    ([500, 131], 64, 8, 1, 128, 256, "random"),  # 512 rows: two row groups
    ([400], 40, 16, 2, 64, 16, "roots"),  # 320 rows: the second group 64
    ([90, 3], 33, 10, 10, 128, 16, "chain"),
    ([4000, 17, 900, 2, 2500, 0, 640], 7, 8, 4, 128, 64, "random"),  # CTAs with several sequences
    ([64] * 30, 2, 16, 8, 64, 32, "chain"),
]


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("ctx,T,H_q,H_kv,d,page,tree", TREES)
def test_trees(kind, ctx, T, H_q, H_kv, d, page, tree):
    c = Case(kind, ctx, T, H_q, H_kv, d, page, tree, seed=T)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_long_context(kind):
    """A context that every CTA has a part of, with later maxima far above the first ones."""
    c = Case(kind, [40000], 6, 8, 2, 128, 64, "random", seed=3)
    if kind == "bf16":
        pages = c.table[0].long()
        for i, t in enumerate(range(3000, 40000, 4099)):  # keys along the queries, each larger than the last
            c.pool.k[pages[t // 64], t % 64] = c.q[0, i % 6, ::4] * (0.2 * i + 0.3)
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_a_single_token_is_a_dense_decode_step(kind):
    c = Case(kind, [300, 77], 1, 8, 4, 128, 32, seed=5)
    out, lse = c.run()
    c.check(out, lse)
    if kind == "kv4":
        from block_sparse_long_index_gb300 import MsaDecodeKv4
        o, l = MsaDecodeKv4(c.pool, 2, c.table.shape[1], 8).dense(c.q[:, 0].contiguous(), c.table, i32([301, 78]), c.scale)
        assert float((o.float() - out[:, 0].float()).abs().max()) < 0.02 and float((l - lse[:, 0]).abs().max()) < 1e-4


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_trees_of_different_lengths(kind):
    tl = [9, 0, 1, 5]
    c = Case(kind, [130, 40, 0, 257], 9, 8, 2, 64, 16, seed=6)
    out, lse = c.run(tree_len=tl)
    assert c.dec.device_status() == 0
    c.check(out, lse, tl)


@pytest.mark.parametrize("T,gs", [(5, 2), (40, 8)])
def test_what_a_node_does_not_see_counts_for_nothing(T, gs):
    """NaN and infinities in drafts beside the branch, in the pages past the tree and in other sequences' pages."""
    ctx = [200, 131]
    c = Case("bf16", ctx, T, 2 * gs, 2, 128, 16, "random", seed=8)
    bad = T - 1  # the last node: no node is below it
    seen = torch.zeros(c.n_pages * 16, dtype=torch.bool, device="cuda")
    t = c.table.long()
    for b in range(2):
        at = torch.arange(ctx[b] + bad, device="cuda")
        seen[t[b, at // 16] * 16 + at % 16] = True
    c.pool.k.flatten(0, 1)[~seen] = math.nan
    c.pool.v.flatten(0, 1)[~seen] = math.inf
    out, lse = c.run()
    for b in range(2):
        k, v = c.values(b, ctx[b] + bad)
        want, wl, A, S = ref.tree_attend(c.q[b, :bad].double(), k, v, ctx[b], c.parents[b][:bad], c.scale)
        sref.check_attention(out[b, :bad].flatten(0, 1), lse[b, :bad].flatten(), want.flatten(0, 1), wl.flatten(), A.flatten(0, 1),
                             S.flatten(), 128, ctx[b] + T)
        assert bool(lse[b, bad].isnan().all()) and bool(out[b, bad].isnan().all())


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_nan_in_the_context_reaches_its_head(kind):
    c = Case(kind, [300, 300], 4, 4, 2, 64, 32, seed=9)
    t = int(c.table[0, 5]) , 7  # token 167 of the first sequence, head 1
    if kind == "bf16":
        c.pool.k[t[0], t[1], 1, 3] = math.nan
    else:
        c.pool.k_scales[t[0], t[1], 1, 0] = 255
    out, lse = c.run()
    assert bool(lse[0, :, 2:].isnan().all()) and bool(out[0, :, 2:].isnan().all())
    assert bool(out[0, :, :2].isfinite().all()) and bool(out[1].isfinite().all())
    c.check(out, lse, only=[1])


def test_scores_of_minus_infinity():
    """A head all of whose scores are -inf: out 0, lse -inf; -inf beside others weighs nothing."""
    c = Case("bf16", [140, 20], 3, 2, 1, 64, 16, "chain", seed=10)
    c.q[:] = c.q.abs() + 0.01
    c.pool.v.copy_(rows(*c.pool.v.shape, seed=11))
    for b in range(2):
        for i in range(c.ctx[b] + 3):
            if b == 0 or i % 3 == 0:
                c.pool.k[c.table[b, i // 16].long(), i % 16] = -math.inf
    out, lse = c.run()
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    assert bool(out[1].isfinite().all()) and bool(lse[1].isfinite().all())
    k, v = c.values(1, 23)
    keep = [i for i in range(23) if i % 3]
    for n in range(3):
        at = [i for i in keep if i <= 20 + n]
        want, wl, A, S = sref.attend(c.q[1, n].double(), k[at, 0], v[at, 0], c.scale)
        sref.check_attention(out[1, n], lse[1, n], want, wl, A, S, 64, 23)


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_bad_pages_parents_and_lengths(kind):
    from block_sparse_long_index_gb300 import msa
    c = Case(kind, [100, 60, 30], 4, 4, 2, 64, 16, "chain", seed=12)
    good, good_lse = (t.clone() for t in c.run())
    for b, at, value in ((0, 2, c.n_pages), (0, 2, -1), (0, 6, -7)):  # in the context, in the context, among the drafts
        keep = int(c.table[b, at])
        c.table[b, at] = value
        out, _ = c.run()
        assert c.dec.device_status() == msa.MSA_ERR_BAD_INDEX
        assert torch.equal(out[1:], good[1:]) and bool(out.isfinite().all())
        c.table[b, at] = 0  # what was read in its place
        same, _ = c.run()
        assert c.dec.device_status() == 0 and torch.equal(same, out)
        c.table[b, at] = keep
    c.parents[1][2] = 2  # its own parent: counts as a root
    out, lse = c.run()
    assert c.dec.device_status() == msa.MSA_ERR_BAD_INDEX
    c.parents[1][2] = -1
    c.check(out, lse)
    c.parents[1][2] = 1
    cap = c.table.shape[1] * 16
    for ctx in ([100, -1, 30], [100, cap - 3, 30]):
        c.ctx = ctx
        out, lse = c.run()
        assert c.dec.device_status() == msa.MSA_ERR_BAD_INDEX
        assert torch.equal(out[::2], good[::2]) and bool((out[1] == 7).all()) and bool((lse[1] == 7).all())
    c.ctx = [100, 60, 30]
    for tl in ([4, -1, 4], [4, 5, 4]):
        out, _ = c.run(tree_len=tl)
        assert c.dec.device_status() == msa.MSA_ERR_BAD_INDEX and torch.equal(out[::2], good[::2]) and bool((out[1] == 7).all())


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_two_calls_at_once_streams_and_graphs(kind):
    from block_sparse_long_index_gb300 import MsaTreeDecode
    a, b = Case(kind, [3000, 10], 8, 8, 2, 128, 64, seed=13), Case(kind, [500, 2000], 30, 16, 2, 128, 32, seed=14)
    want = [tuple(t.clone() for t in c.run()) for c in (a, b)]
    runs = [(c, MsaTreeDecode(c.pool, c.B, c.T, c.table.shape[1], c.H_q), torch.cuda.Stream(), i32(c.ctx), i32(c.parents)) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, s, ctx, par in runs:
            d(c.q, c.table, ctx, par, None, c.scale, stream=s)
    torch.cuda.synchronize()
    for (c, d, *_), w in zip(runs, want):
        assert torch.equal(d.out, w[0]) and torch.equal(d.lse, w[1])  # equal calls give equal bits
    c, d, _, ctx, par = runs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d(c.q, c.table, ctx, par, None, c.scale)
    ctx.copy_(i32([2000, 333]))
    c.ctx = [2000, 333]
    counts = [-(-(n + c.T) // 64) for n in [3000, 3000]]
    c.table[1, :counts[1]] = torch.randperm(c.n_pages, device="cuda")[:counts[1]].int()
    d.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check(d.out, d.lse)


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_pool_past_32_bit_offsets(kind):
    """The last pages of a pool beyond 2^32 bytes (4 bits: of codes)."""
    from block_sparse_long_index_gb300 import Kv4Pool, KvPool
    c = Case(kind, [200], 4, 16, 8, 128, 128, seed=15)
    row = 8 * 128 * 2 if kind == "bf16" else 8 * 64
    n_pages = (1 << 32) // (128 * row) + 16
    big = []
    for t in c.pool.tensors():
        x = torch.zeros((n_pages,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        x[-c.n_pages:] = t
        big.append(x)
    c.table = torch.where(c.table >= 0, c.table + (n_pages - c.n_pages), c.table)
    c.n_pages, c.pool = n_pages, (KvPool if kind == "bf16" else Kv4Pool)(*big)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse)


def test_many_sequences():
    """More sequences than the context kernel has threads, some empty."""
    r = np.random.default_rng(16)
    ctx = [int(x) for x in r.integers(0, 40, 2000)]
    c = Case("bf16", ctx, 2, 2, 1, 64, 16, "chain", seed=16)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse, only=[0, 1, 2, 700, 767, 768, 769, 1500, 1998, 1999] + [int(i) for i in r.integers(0, 2000, 40)])


def test_tree_refusals():
    c = Case("bf16", [40, 30], 3, 4, 2, 64, 16, seed=17)
    c.run()
    d, ctx, par = c.dec, i32(c.ctx), i32(c.parents)
    for bad in (dict(q=c.q[:1]), dict(q=c.q.float()), dict(q=c.q.transpose(1, 2)), dict(page_table=c.table[:, :1]), dict(ctx_len=ctx.long()),
                dict(parents=par[:, :2]), dict(parents=par.cpu()), dict(tree_len=i32([1]))):
        with pytest.raises(ValueError):
            d(**{**dict(q=c.q, page_table=c.table, ctx_len=ctx, parents=par), **bad})


FORMS = [  # rows a K/V head about 8, 16 and 32, where the 4-bit cache's kernel changes its form, by K/V heads
    ([500, 0, 31, 16, 15, 700], 8, 8, 8, 128, 16, "random"),
    ([300, 17], 9, 5, 5, 128, 48, "wide"),
    ([777, 1, 2000], 4, 28, 7, 64, 32, "random"),
    ([250, 33], 17, 3, 3, 128, 16, "chain"),
    ([1200, 5], 8, 16, 4, 64, 80, "random"),
    ([90, 4000], 2, 16, 2, 128, 64, "chain"),
    ([2500], 31, 2, 2, 64, 16, "random"),
    ([1, 47, 48, 49], 8, 1, 1, 64, 16, "random"),
    ([3000, 100], 3, 4, 1, 128, 32, "wide"),
    ([640], 32, 8, 8, 128, 128, "random"),
    ([640, 9], 33, 8, 8, 128, 128, "random"),
    ([200, 321], 2, 18, 9, 64, 16, "chain"),
]


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
@pytest.mark.parametrize("ctx,T,H_q,H_kv,d,page,tree", FORMS)
def test_forms(kind, ctx, T, H_q, H_kv, d, page, tree):
    c = Case(kind, ctx, T, H_q, H_kv, d, page, tree, seed=20 + T)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("T,gs", [(3, 2), (7, 2), (5, 4), (12, 8)])
def test_groups_that_hold_nan_in_the_4_bit_context(T, gs):
    """A NaN group of K makes its head's rows NaN, one of V its channels; past the context neither counts."""
    c = Case("kv4", [300, 75], T, 2 * gs, 2, 128, 16, "chain", seed=21)
    c.pool.k_scales[c.table[0, 9].long(), 3, 1, 2] = 255  # token 147, head 1
    c.pool.v_scales[c.table[0, 4].long(), 15, 0, 1] = 255  # token 79, head 0, channels 32 .. 63
    for p, at in ((c.table[1, 4], 11 + T), (c.table[0, 18], 12 + T)):  # behind the last node, in its page
        if at < 16:
            c.pool.k_scales[p.long(), at:] = 255
            c.pool.v_scales[p.long(), at:] = 255
    out, lse = c.run()
    assert bool(lse[0, :, gs:].isnan().all()) and bool(out[0, :, gs:].isnan().all())
    assert bool(lse[0, :, :gs].isfinite().all()) and bool(out[0, :, :gs, 32:64].isnan().all())
    assert bool(out[0, :, :gs, :32].isfinite().all()) and bool(out[0, :, :gs, 64:].isfinite().all())
    c.check(out, lse, only=[1])


def test_many_rows_over_a_4_bit_pool_past_32_bit_offsets():
    from block_sparse_long_index_gb300 import Kv4Pool
    c = Case("kv4", [200], 24, 16, 8, 128, 128, seed=22)
    n_pages = (1 << 32) // (128 * 8 * 64) + 16
    big = []
    for t in c.pool.tensors():
        x = torch.zeros((n_pages,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        x[-c.n_pages:] = t
        big.append(x)
    c.table = torch.where(c.table >= 0, c.table + (n_pages - c.n_pages), c.table)
    c.n_pages, c.pool = n_pages, Kv4Pool(*big)
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse)


@pytest.mark.parametrize("T,H_q", [(2, 4), (24, 8)])
def test_a_long_4_bit_context(T, H_q):
    """Every CTA has a part of one sequence; keys much larger than the ones before move the maxima late."""
    c = Case("kv4", [50000], T, H_q, 2, 128, 64, "random", seed=23)
    pages = c.table[0].long()
    for i, t in enumerate(range(3000, 50000, 6007)):
        c.pool.k_scales[pages[t // 64], t % 64] = 160 + 2 * i
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse)


def test_many_sequences_in_4_bits():
    """More sequences than a CTA has threads, some empty."""
    r = np.random.default_rng(24)
    ctx = [int(x) for x in r.integers(0, 40, 900)]
    for T, H_q in ((2, 2), (10, 8)):
        c = Case("kv4", ctx, T, H_q, 2, 64, 16, "chain", seed=24)
        out, lse = c.run()
        assert c.dec.device_status() == 0
        c.check(out, lse, only=[0, 1, 2, 255, 256, 257, 511, 898, 899] + [int(i) for i in r.integers(0, 900, 12)])


def test_room_for_more_spans_than_an_int_counts():
    """A table whose width alone, times the sequences, asks for the coarser split of the 4-bit form's list."""
    r = np.random.default_rng(25)
    ctx = [int(x) for x in r.integers(0, 300, 1024)]
    c = Case("kv4", ctx, 2, 2, 1, 64, 256, "chain", seed=25)
    wide = torch.full((c.B, 1 << 18), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    out, lse = c.run()
    assert c.dec.device_status() == 0
    c.check(out, lse, only=[0, 1, 511, 512, 1022, 1023] + [int(i) for i in r.integers(0, 1024, 12)])
