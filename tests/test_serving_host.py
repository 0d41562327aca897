"""Refusals of the serving calls (validated before any launch) and pins of the 64-bit references; no GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from test_capi_host import lib  # noqa: F401  (the library as a fixture)

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40


def test_dense_prefill_refusals(lib):  # noqa: F811
    f = lib.raw().msa_dense_prefill_varlen

    def call(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, S=2, N=100, H_q=8, H_kv=2, d=128, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=0):
        return f(q, k, v, cu, S, N, H_q, H_kv, d, scale, out, lse, ws, wb, None)

    assert call() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(lse=None), dict(S=0),
                dict(N=0), dict(H_q=0), dict(H_kv=0), dict(d=0), dict(H_q=7), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD),
                dict(lse=ctypes.c_void_p(2)), dict(ws=None), dict(ws=ODD, wb=BIG)):
        assert call(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in (dict(d=96), dict(H_q=32), dict(H_q=6), dict(H_kv=65, H_q=65), dict(N=(1 << 24) + 1)):
        assert call(**bad) == lib.MSA_ERR_UNSUPPORTED, bad
    assert lib.msa_dense_prefill_varlen_workspace(1000, 3, 8, 1, 128) > 256
    assert lib.msa_dense_prefill_varlen_workspace(0, 3, 8, 1, 128) == 256


def pool_of(lib, **kw):  # noqa: F811
    a = dict(k_codes=1 << 20, k_scales=1 << 20, v_codes=1 << 20, v_scales=1 << 20, n_pages=4, page_size=16, H_kv=2, d=64)
    a.update(kw)
    return lib.msa_kv4_pool_t(*a.values())


BAD_POOLS = [dict(k_codes=0), dict(k_scales=0), dict(v_codes=0), dict(v_scales=0), dict(n_pages=0), dict(page_size=0),
             dict(page_size=24), dict(H_kv=0), dict(d=0), dict(k_codes=(1 << 20) + 8), dict(v_scales=(1 << 20) + 4)]
OTHER_POOLS = [dict(d=96), dict(H_kv=65), dict(n_pages=1 << 31)]


def test_kv4_row_refusals(lib):  # noqa: F811
    raw = lib.raw()

    def store(pool=None, k=FAKE, v=FAKE, N=3, cu=FAKE, S=1, pos=FAKE, table=FAKE, mp=2, ws=FAKE, wb=0):
        p = pool_of(lib) if pool is None else pool
        return raw.msa_kv4_store(k, v, N, cu, S, pos, table, mp, ctypes.byref(p), ws, wb, None)

    def load(pool=None, k=FAKE, v=FAKE, N=3, cu=FAKE, S=1, pos=FAKE, table=FAKE, mp=2, ws=FAKE, wb=0):
        p = pool_of(lib) if pool is None else pool
        return raw.msa_kv4_load(ctypes.byref(p), N, cu, S, pos, table, mp, k, v, ws, wb, None)

    for f in (store, load):
        assert f() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        for bad in (dict(k=None), dict(v=None), dict(cu=None), dict(pos=None), dict(table=None), dict(N=0), dict(S=0),
                    dict(mp=0), dict(k=ODD), dict(ws=None), dict(cu=ctypes.c_void_p(2))):
            assert f(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in BAD_POOLS:
            assert f(pool_of(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        for bad in OTHER_POOLS:
            assert f(pool_of(lib, **bad)) == lib.MSA_ERR_UNSUPPORTED, bad
        assert f(mp=1 << 28) == lib.MSA_ERR_UNSUPPORTED  # positions past 31 bits
    assert raw.msa_kv4_store(FAKE, FAKE, 3, FAKE, 1, FAKE, FAKE, 2, None, FAKE, BIG, None) == lib.MSA_ERR_INVALID_ARGUMENT


def test_kv4_decode_refusals(lib):  # noqa: F811
    raw = lib.raw()

    def dense(pool=None, q=FAKE, table=FAKE, mp=2, ctx=FAKE, B=2, H_q=8, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=0):
        p = pool_of(lib) if pool is None else pool
        return raw.msa_dense_decode_paged_kv4(q, ctypes.byref(p), table, mp, ctx, B, H_q, scale, out, lse, ws, wb, None)

    assert dense() == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    assert dense(lse=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL  # lse may be left out
    for bad in (dict(q=None), dict(table=None), dict(ctx=None), dict(out=None), dict(B=0), dict(H_q=0), dict(H_q=5),
                dict(scale=0.0), dict(scale=math.nan), dict(q=ODD), dict(out=ODD), dict(ws=None), dict(mp=0)):
        assert dense(**bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in BAD_POOLS:
        assert dense(pool_of(lib, **bad)) == lib.MSA_ERR_INVALID_ARGUMENT, bad
    for bad in OTHER_POOLS:
        assert dense(pool_of(lib, **bad)) == lib.MSA_ERR_UNSUPPORTED, bad
    assert dense(H_q=32) == lib.MSA_ERR_UNSUPPORTED and dense(H_q=6) == lib.MSA_ERR_UNSUPPORTED

    for f in (raw.msa_decode_paged_kv4, raw.msa_decode_paged_kv4_fp8):
        def step(shape, pool=None, q=FAKE, qi=FAKE, ki=FAKE, mp=8, B=2, scale=0.1, wb=0, f=f):
            p = pool_of(lib) if pool is None else pool
            return f(q, qi, ki, ctypes.byref(p), FAKE, mp, FAKE, B, ctypes.byref(shape), scale, FAKE, None, None, FAKE, wb,
                     None)
        good = lib.shape(128, 8, 2, 64, 64, 64, 2)
        assert step(good) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
        for bad in (dict(q=None), dict(qi=None), dict(ki=None), dict(B=0), dict(scale=-1.0), dict(mp=9)):
            assert step(good, **bad) == lib.MSA_ERR_INVALID_ARGUMENT, bad
        assert step(lib.shape(128, 8, 4, 64, 64, 64, 2)) == lib.MSA_ERR_INVALID_ARGUMENT  # not the pool's heads
        assert step(lib.shape(128, 8, 2, 128, 64, 64, 2)) == lib.MSA_ERR_INVALID_ARGUMENT
        assert step(lib.shape(128, 8, 2, 64, 48, 64, 2)) == lib.MSA_ERR_UNSUPPORTED
    assert raw.msa_decode_paged_kv4_fp8(FAKE, FAKE, FAKE, ctypes.byref(pool_of(lib)), FAKE, 8, FAKE, 2,
                                        ctypes.byref(lib.shape(128, 8, 2, 64, 32, 64, 2)), 0.1, FAKE, None, None, FAKE,
                                        BIG, None) == lib.MSA_ERR_UNSUPPORTED


def test_page_refusals(lib):  # noqa: F811
    raw = lib.raw()

    def tables(**kw):
        a = dict(table=1 << 20, ctx=1 << 20, refs=1 << 20, max_pages=4, n_pages=10, n_seqs=3, page=16)
        a.update(kw)
        return lib.msa_pages_t(*a.values())

    one = lib.page_pools([(1 << 20, 64)])
    calls = {
        "reserve": lambda p, n=2, a=FAKE, b=FAKE, ws=FAKE, wb=0: raw.msa_pages_reserve(ctypes.byref(p), a, b, n, ws, wb, None),
        "fork": lambda p, n=2, a=FAKE, b=FAKE, ws=FAKE, wb=0: raw.msa_pages_fork(ctypes.byref(p), a, b, n, one, 1, ws, wb, None),
        "free": lambda p, n=2, a=FAKE, b=FAKE, ws=FAKE, wb=0: raw.msa_pages_free(ctypes.byref(p), a, n, ws, wb, None),
    }
    for name, f in calls.items():
        assert f(tables()) == lib.MSA_ERR_WORKSPACE_TOO_SMALL, name
        for bad in (dict(table=0), dict(ctx=0), dict(refs=0), dict(max_pages=0), dict(n_pages=0), dict(n_seqs=0),
                    dict(page=0), dict(page=20), dict(refs=(1 << 20) + 2)):
            assert f(tables(**bad)) == lib.MSA_ERR_INVALID_ARGUMENT, (name, bad)
        for bad in (dict(n_pages=1 << 27), dict(max_pages=1 << 27)):
            assert f(tables(**bad)) == lib.MSA_ERR_UNSUPPORTED, (name, bad)
        assert f(tables(), n=-1) == lib.MSA_ERR_INVALID_ARGUMENT
        assert f(tables(), n=4097) == lib.MSA_ERR_UNSUPPORTED
        assert f(tables(), a=None) == lib.MSA_ERR_INVALID_ARGUMENT
        assert f(tables(), ws=None) == lib.MSA_ERR_INVALID_ARGUMENT
        assert f(tables(), n=0, a=None, b=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    p = tables()

    def compact(pools=one, n=1, map_=FAKE, live=FAKE, wb=0):
        return raw.msa_pages_compact(ctypes.byref(p), pools, n, map_, live, FAKE, wb, None)

    assert compact() == lib.MSA_ERR_WORKSPACE_TOO_SMALL and compact(map_=None, live=None) == lib.MSA_ERR_WORKSPACE_TOO_SMALL
    assert compact(n=-1) == lib.MSA_ERR_INVALID_ARGUMENT and compact(pools=None) == lib.MSA_ERR_INVALID_ARGUMENT
    assert compact(pools=lib.page_pools([(1 << 20, 64)] * 9), n=9) == lib.MSA_ERR_UNSUPPORTED
    for entry in ((0, 64), (1 << 20, 0), (1 << 20, 40), ((1 << 20) + 8, 64)):
        assert compact(pools=lib.page_pools([entry])) == lib.MSA_ERR_INVALID_ARGUMENT, entry
    assert compact(map_=ctypes.c_void_p(2)) == lib.MSA_ERR_INVALID_ARGUMENT
    assert "free pages" in lib.msa_status_string(lib.MSA_ERR_NO_PAGES)


# ---------------------------------------------------------------- the references themselves
def test_format_pins():
    sv = ref.scale_values()
    assert sv[0] == 2.0 ** -20 and sv[8 * 20] == 1.0 and sv[254] == 3584.0 and np.all(np.diff(sv) > 0)
    x = np.array([7.0, 3.5, -7.0, 0.5, 1.5, 2.5, -0.5, 0.0] + [0.0] * 8 * 7)  # d = 64: scale 1 in the first group
    c, s = ref.quantize(x)
    assert s[0] == 160 and c[:8].tolist() == [15, 12, 1, 8, 10, 10, 8, 8]  # 3.5 -> 4, 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    assert s[1] == 0 and (c[16:] == 8).all()
    assert np.array_equal(ref.unpack(ref.pack(c)), c)
    w = ref.pack(np.arange(8).repeat(8).reshape(8, 8).T.reshape(-1)[None])[0, :4]  # channels 0..7 -> their own numbers
    assert [int(b) for b in w] == [0 | 2 << 4, 4 | 6 << 4, 1 | 3 << 4, 5 | 7 << 4]
    # every value is exact in bf16
    vals = ((np.arange(16) - 8)[:, None] * sv[None]).ravel()
    t = torch.from_numpy(vals)
    assert torch.equal(t.to(torch.bfloat16).double(), t)


def test_attention_pins():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(9, 4, 64, generator=g).to(torch.bfloat16) for _ in range(3))
    out, lse, A, S = ref.dense_prefill(q, k, v, [4, 0, 5], 0.125)
    for h in range(4):
        want = torch.nn.functional.scaled_dot_product_attention(*[t[4:, h].double()[None] for t in (q, k, v)], is_causal=True,
                                                                scale=0.125)
        assert torch.allclose(out[4:, h], want[0], atol=1e-12)
    assert torch.allclose(lse[0], (q[0].double() * k[0].double()).sum(-1) * 0.125)
    o, l, _, _ = ref.attend(q[8].double(), k[4:, 2].double(), v[4:, 2].double(), 0.125)
    assert torch.allclose(o[2], out[8, 2]) and torch.allclose(l[2], lse[8, 2])


def test_pages_pins():
    p = ref.PagesRef(4, 4, 6, 16)
    assert p.reserve([1, 0], [20, 16]) and p.table[1] == [0, 1] and p.table[0] == [2]
    assert p.fork([1], [2]) and p.table[2] == [0, 3] and p.refs == [2, 1, 1, 1, 0, 0] and p.data[3] == 1
    p.free([1, 0])
    assert p.refs == [1, 0, 0, 1, 0, 0]
    assert p.compact() == ([0, -1, -1, 1, -1, -1], 2) and p.table[2] == [0, 1] and p.data[1] == 1
    assert not p.reserve([0], [16 * 5])


def test_limits_of_packed_calls(lib):  # noqa: F811
    """The number of sequences stays where sums of two of them fit an int."""
    raw, S = lib.raw(), 1 << 24
    p = pool_of(lib)
    for n, want in ((S, lib.MSA_ERR_WORKSPACE_TOO_SMALL), (S + 1, lib.MSA_ERR_UNSUPPORTED),
                    ((1 << 31) - 1, lib.MSA_ERR_UNSUPPORTED)):
        assert raw.msa_dense_prefill_varlen(FAKE, FAKE, FAKE, FAKE, n, 1000, 8, 2, 128, 0.1, FAKE, FAKE, FAKE, 0, None) == want
        assert raw.msa_kv4_store(FAKE, FAKE, 3, FAKE, n, FAKE, FAKE, 2, ctypes.byref(p), FAKE, 0, None) == want
        assert raw.msa_kv4_load(ctypes.byref(p), 3, FAKE, n, FAKE, FAKE, 2, FAKE, FAKE, FAKE, 0, None) == want
    assert lib.msa_dense_prefill_varlen_workspace(1000, S, 8, 2, 128) > 4 * S
    assert lib.msa_dense_prefill_varlen_workspace(1000, S + 1, 8, 2, 128) == 256
    assert raw.msa_kv4_store(FAKE, FAKE, 1 << 31, FAKE, 1, FAKE, FAKE, 2, ctypes.byref(p), FAKE, 0, None) == lib.MSA_ERR_UNSUPPORTED


def test_tensors_of_another_device(monkeypatch):
    """The serving classes refuse tensors and calls of another device than their own (stand-ins for CUDA tensors)."""
    from block_sparse_long_index_gb300 import Kv4Pool, PagedCache, api

    class On:
        def __init__(self, dev, shape=(3,), dtype=torch.int32, contiguous=True):
            self.dev, self.shape, self.dtype, self.contiguous = dev, torch.Size(shape), dtype, contiguous

        def get_device(self):
            return self.dev

        def is_contiguous(self):
            return self.contiguous

    api._check_tensor("x", On(1), torch.int32, (3,), 1)
    api._check_tensor("x", On(1), torch.int32, (3,))
    for t, dev, words in ((On(1), 0, "cuda:1"), (On(-1), -1, "contiguous CUDA"), (On(-1), None, "contiguous CUDA"),
                          (On(0, dtype=torch.int64), 0, "contiguous CUDA int32"), (On(0, (4,)), 0, "shape"),
                          (On(0, contiguous=False), 0, "contiguous")):
        with pytest.raises(ValueError, match=words):
            api._check_tensor("x", t, torch.int32, (3,), dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert api._device(On(1)) == 1
    with pytest.raises(ValueError, match="cuda:0"):
        api._device(On(0))
    with pytest.raises(ValueError, match="CUDA"):
        PagedCache(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="CUDA"):
        Kv4Pool(*[torch.zeros(2, 16, 1, n, dtype=torch.uint8) for n in (32, 4, 32, 4)])


def stand_in_pool(dev, monkeypatch):
    """A pool of device `dev` for MsaDecodeKv4, and the devices of what is allocated from here on (on `meta`)."""
    class Codes:
        device = torch.device("cuda", dev)

        def get_device(self):
            return dev

    class Pool:
        k_codes, n_pages, page_size, H_kv, d = Codes(), 4, 16, 2, 64

    made, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: made.append(torch.device(device)) or empty(*a, device="meta", **k))
    return Pool(), made


@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda", 0)])
def test_decode_kv4_allocates_beside_its_pool(monkeypatch, lib, device):  # noqa: F811
    """The workspace and the outputs lie on the pool's device, whatever device is current."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    pool, made = stand_in_pool(0, monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    MsaDecodeKv4(pool, 2, 3, 8, d_I=64, Bk=64, k=2, device=device)
    assert len(made) >= 4 and set(made) == {torch.device("cuda", 0)}


@pytest.mark.parametrize("device", ["cuda:1", "cpu", torch.device("cuda", 7)])
def test_decode_kv4_refuses_another_device(monkeypatch, lib, device):  # noqa: F811
    from block_sparse_long_index_gb300 import MsaDecodeKv4
    pool, made = stand_in_pool(0, monkeypatch)
    with pytest.raises(ValueError, match="cuda:0"):
        MsaDecodeKv4(pool, 2, 3, 8, device=device)
    assert not made
