"""The speculative-decoding calls without a GPU: refusals (validated before any launch), frequency tables, and pins of the
64-bit references."""
import ctypes
import math

import numpy as np
import pytest
import torch

import draft_ref as ref
from test_capi_host import lib  # noqa: F401  (the library as a fixture)
from test_serving_host import BAD_POOLS, BIG, FAKE, ODD, OTHER_POOLS, pool_of

HALF = ctypes.c_void_p((1 << 20) + 2)


def rope_of(lib, **kw):  # noqa: F811
    a = dict(turns=1 << 20, rot=64, interleaved=0, factor=1.0)
    a.update(kw)
    return lib.msa_rope_t(*a.values())


def test_rope_refusals(lib):  # noqa: F811
    def call(rope="good", x=FAKE, xs=512, y=FAKE, ys=512, N=3, H=4, d=128, f32=0, pos=FAKE):
        r = rope_of(lib) if rope == "good" else rope
        return lib.raw().msa_rope(x, xs, y, ys, N, H, d, f32, pos, None if r is None else ctypes.byref(r), 0, None)

    for bad in (dict(x=None), dict(y=None), dict(pos=None), dict(N=0), dict(H=0), dict(d=0), dict(x=ODD), dict(y=ODD), dict(pos=HALF),
                dict(xs=511), dict(xs=504), dict(ys=516), dict(ys=511, f32=1), dict(ys=514, f32=1), dict(xs=1024), dict(rope=None)):
        assert call(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(turns=0), dict(turns=(1 << 20) + 4), dict(rot=0), dict(rot=144), dict(factor=math.inf), dict(factor=math.nan)):
        assert call(rope_of(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    assert call(rope_of(lib, rot=24)) == lib.MSA_ERR_UNSUPPORTED
    for d in (16, 48, 96, 512):
        assert call(d=d, xs=8192, ys=8192) == lib.MSA_ERR_UNSUPPORTED


def append_of(lib, **kw):  # noqa: F811
    P = 1 << 20
    a = dict(q=P, k=P, v=P, q_idx=P, k_idx=P, q_stride=512, k_stride=128, v_stride=128, q_idx_stride=128, k_idx_stride=64, q_out=2 * P,
             q_idx_out=2 * P, k_idx_pool=P, positions=0, H_q=8, d_I=64, idx_f8=0, idx_scale=1.0)
    a.update(kw)
    return lib.msa_append_t(*a.values())


def kv_pool_of(lib, **kw):  # noqa: F811
    a = dict(k=1 << 20, v=1 << 20, n_pages=4, page_size=16, H_kv=2, d=64)
    a.update(kw)
    return lib.msa_kv_pool_t(*a.values())


BAD_KV = [dict(k=0), dict(v=0), dict(n_pages=0), dict(page_size=0), dict(page_size=24), dict(H_kv=0), dict(d=0), dict(k=(1 << 20) + 8)]


def test_append_refusals(lib):  # noqa: F811
    raw = lib.raw()
    for f, make, bad_pools in ((raw.msa_append_paged, kv_pool_of, BAD_KV), (raw.msa_append_paged_kv4, pool_of, BAD_POOLS)):
        def call(rows="good", pool=None, rope="good", rope_idx="good", N=3, cu=FAKE, S=1, pos=FAKE, table=FAKE, mp=2, ws=FAKE, wb=0,
                 f=f, make=make):
            rows = append_of(lib) if rows == "good" else rows
            pool = make(lib) if pool is None else pool
            ref_of = lambda r: None if r is None else ctypes.byref(rope_of(lib) if r == "good" else r)  # noqa: E731
            return f(None if rows is None else ctypes.byref(rows), N, cu, S, pos, table, mp, ctypes.byref(pool), ref_of(rope),
                     ref_of(rope_idx), ws, wb, None)

        assert call() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        assert call(rope=None, rope_idx=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        for ok in (dict(q=0), dict(k_idx=0), dict(q_idx=0), dict(q_stride=1024), dict(q_out=1 << 20), dict(idx_f8=1)):
            assert call(append_of(lib, **ok)) == lib.MSA_ERR_WORKSPACE_TOO_SMALL, ok
        for bad in (dict(k=0), dict(v=0), dict(k=(1 << 20) + 8), dict(k_stride=120), dict(v_stride=132), dict(q_out=0),
                    dict(q_stride=508), dict(q_stride=1024, q_out=1 << 20), dict(q_out=(1 << 20) + 8), dict(H_q=0), dict(k_idx_pool=0), dict(q_idx_out=0), dict(d_I=0),
                    dict(k_idx_stride=32), dict(positions=(1 << 20) + 2), dict(idx_f8=1, idx_scale=0.0),
                    dict(idx_f8=1, idx_scale=math.inf), dict(idx_f8=1, q_idx_out=1 << 20)):
            assert call(append_of(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(d_I=48), dict(H_q=1024, q_stride=65536)):
            assert call(append_of(lib, **bad)) == lib.MSA_ERR_UNSUPPORTED, bad
        for bad in (dict(rows=None), dict(N=0), dict(S=0), dict(cu=None), dict(pos=None), dict(table=None), dict(mp=0), dict(cu=HALF),
                    dict(ws=None), dict(rope=rope_of(lib, rot=80)), dict(rope_idx=rope_of(lib, rot=128))):
            assert call(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        assert call(append_of(lib, k_idx=0, q_idx=0)) == lib.MSA_ERR_INVALID_ARGUMENT  # index frequencies without index rows
        assert call(append_of(lib, k_idx=0, q_idx=0), rope_idx=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        assert call(rope=rope_of(lib, rot=40)) == lib.MSA_ERR_UNSUPPORTED
        for bad in bad_pools:
            assert call(pool=make(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in OTHER_POOLS:
            assert call(pool=make(lib, **bad)) == lib.MSA_ERR_UNSUPPORTED, bad
        assert call(mp=1 << 28) == lib.MSA_ERR_UNSUPPORTED


def test_tree_refusals(lib):  # noqa: F811
    raw = lib.raw()
    for f, make, bad_pools in ((raw.msa_tree_decode_paged, kv_pool_of, BAD_KV), (raw.msa_tree_decode_paged_kv4, pool_of, BAD_POOLS)):
        def call(pool=None, q=FAKE, table=FAKE, mp=2, ctx=FAKE, tl=None, par=FAKE, B=2, T=5, H_q=8, scale=0.1, out=FAKE, lse=None, ws=FAKE,
                 wb=0, f=f, make=make):
            pool = make(lib) if pool is None else pool
            return f(q, ctypes.byref(pool), table, mp, ctx, tl, par, B, T, H_q, scale, out, lse, ws, wb, None)

        assert call() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        for bad in (dict(q=None), dict(table=None), dict(ctx=None), dict(par=None), dict(out=None), dict(mp=0), dict(B=0), dict(T=0),
                    dict(H_q=0), dict(H_q=5), dict(scale=0.0), dict(scale=math.nan), dict(q=ODD), dict(out=ODD), dict(tl=HALF), dict(lse=HALF), dict(par=HALF), dict(ws=None),
                    dict(ws=ODD, wb=BIG)):
            assert call(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in (dict(T=65), dict(H_q=32), dict(H_q=6), dict(B=(1 << 20) + 1)):
            assert call(**bad) == lib.MSA_ERR_UNSUPPORTED, bad
        for bad in bad_pools:
            assert call(make(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in OTHER_POOLS:
            assert call(make(lib, **bad)) == lib.MSA_ERR_UNSUPPORTED, bad
    assert raw.msa_tree_decode_paged(FAKE, ctypes.byref(kv_pool_of(lib, n_pages=1 << 27)), FAKE, 2, FAKE, None, FAKE, 2, 5, 8, 0.1, FAKE,
                                     None, FAKE, BIG, None) == lib.MSA_ERR_UNSUPPORTED  # 2^31 tokens
    assert lib.msa_tree_decode_workspace(2, 5, 8, 2, 64) > 256 and lib.msa_tree_decode_workspace(0, 5, 8, 2, 64) == 256


def test_verify_and_accept_refusals(lib):  # noqa: F811
    raw = lib.raw()

    def call(p=FAKE, q=FAKE, tok=FAKE, par=FAKE, tl=None, u=FAKE, ul=FAKE, B=2, T=5, V=100, path=FAKE, n=FAKE, nxt=FAKE, ws=FAKE, wb=0):
        return raw.msa_verify_tree(p, q, tok, par, tl, u, ul, B, T, V, path, n, nxt, ws, wb, None)

    assert call() == lib.MSA_ERR_WORKSPACE_TOO_SMALL and call(q=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(p=None), dict(tok=None), dict(par=None), dict(u=None), dict(ul=None), dict(path=None), dict(n=None), dict(nxt=None),
                dict(B=0), dict(T=0), dict(V=0), dict(p=ODD), dict(q=ODD), dict(tok=HALF), dict(tl=HALF), dict(nxt=HALF), dict(ws=None)):
        assert call(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(T=65), dict(V=1 << 31), dict(B=(1 << 20) + 1)):
        assert call(**bad) == lib.MSA_ERR_UNSUPPORTED, bad

    def accept(seqs=FAKE, base=FAKE, path=FAKE, n_path=FAKE, n=2, T=5, page_bytes=512, n_pools=1, ws=FAKE, wb=0, page=16):
        pages = lib.msa_pages_t(1 << 20, 1 << 20, 1 << 20, 4, 10, 3, page)
        pools = lib.page_pools([(1 << 20, page_bytes)])
        return raw.msa_pages_accept(ctypes.byref(pages), seqs, base, path, n_path, n, T, pools, n_pools, ws, wb, None)

    assert accept() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(seqs=None), dict(base=None), dict(path=None), dict(n_path=None), dict(n=-1), dict(T=0), dict(path=HALF),
                dict(page_bytes=520), dict(page_bytes=80, page=32), dict(ws=None), dict(n_pools=-1), dict(page=24)):
        assert accept(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(T=65), dict(n=4097), dict(n_pools=9)):
        assert accept(**bad) == lib.MSA_ERR_UNSUPPORTED, bad


# ---------------------------------------------------------------- frequencies
def test_frequency_tables():
    from block_sparse_long_index_gb300 import rope_frequencies
    f = rope_frequencies(64, 10000.0)
    assert f[0] == 1.0 and len(f) == 32 and math.isclose(f[16], 10000.0 ** -0.5)
    assert rope_frequencies(64, 10000.0, "linear", 4.0) == [x / 4 for x in f]
    b = rope_frequencies(64, 10000.0, "base", 8.0)
    assert b[0] == 1.0 and math.isclose(b[-1], f[-1] / 8.0, rel_tol=1e-12)
    p = rope_frequencies(128, 10000.0, "parts", 4.0, original_len=4096)
    f = rope_frequencies(128, 10000.0)
    turns = [4096 * x / (2 * math.pi) for x in f]  # within the training length
    assert all(a == x for a, x, t in zip(p, f, turns) if t > 2 * 32)
    assert all(math.isclose(a, x / 4) for a, x, t in zip(p, f, turns) if t < 0.5)
    assert all(x / 4 * (1 - 1e-12) <= a <= x for a, x in zip(p, f)) and all(a > b for a, b in zip(p, p[1:]))
    for bad in (dict(rot=7), dict(rot=0), dict(base=1.0), dict(factor=0.5), dict(scaling="odd"), dict(scaling="parts"),
                dict(rot=2, scaling="base")):
        with pytest.raises(ValueError):
            rope_frequencies(**{"rot": 64, **bad})


def test_turns_are_the_nearest_fixed_point():
    from fractions import Fraction

    from block_sparse_long_index_gb300.api import _turns
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    for f in (1.0, 0.1, 1e-4, 3.7e-9, 2.5, 1234.5, 0.0, -0.25):
        exact = Fraction(f) / (2 * pi) * 2 ** 64
        t = _turns(f)
        assert -(1 << 63) <= t < 1 << 63
        off = (exact - t) % (1 << 64)
        assert min(off, (1 << 64) - off) <= Fraction(1, 2), f
    for bad in (math.inf, math.nan):
        with pytest.raises(ValueError):
            _turns(bad)


# ---------------------------------------------------------------- the references themselves
def test_turned_rows_keep_their_products():
    """A rotation keeps lengths, its inverse undoes it, and products depend on the distance of positions alone."""
    r = np.random.default_rng(0)
    q, k = (torch.tensor(r.standard_normal((1, 1, 32))) for _ in range(2))
    freqs = [10000.0 ** (-2 * i / 16) for i in range(8)]
    for inter in (False, True):
        a = ref.turn(q, [1000007], freqs, inter)
        assert torch.allclose(a.norm(), q.norm(), rtol=1e-14, atol=0)
        assert torch.allclose(ref.turn(a, [1000007], freqs, inter, inverse=True), q, rtol=0, atol=1e-13)
        x = (ref.turn(q, [57], freqs, inter) * ref.turn(k, [17], freqs, inter)).sum()
        y = (ref.turn(q, [1000040], freqs, inter) * ref.turn(k, [1000000], freqs, inter)).sum()
        assert abs(float(x - y)) < 1e-12


@pytest.mark.parametrize("children", [1, 2, 3])
def test_verification_follows_the_target(children):
    """Whatever the drafts are drawn from, the token after node 0 (an accepted child's, or the next one) is distributed as
    the target says: frequencies over all of a grid of random numbers, against p."""
    r = np.random.default_rng(children)
    V = 5
    p, q = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    n = 60000
    counts = np.zeros(V)
    P, Q = np.stack([p] * (children + 1)), np.stack([q] * (children + 1))
    for _ in range(n):
        tokens = [0] + list(r.choice(V, size=children, p=q))
        path, nxt, _ = ref.verify(P, Q, tokens, [-1] + [0] * children, r.random(children + 1), r.random())
        counts[tokens[path[1]] if len(path) > 1 else nxt] += 1
    sigma = np.sqrt(p * (1 - p) / n)
    assert (np.abs(counts / n - p) < 5 * sigma).all(), (counts / n, p)  # five standard deviations, five tokens: 3e-6
