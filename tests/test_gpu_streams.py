"""Objects that are made while the current stream is busy and first used on another one."""
import pytest
import torch

from test_gpu_kv4 import i32
from test_gpu_rope import rows

pytestmark = pytest.mark.gpu


@pytest.fixture
def late():
    """A stream, and a function that gives the current one some 20 ms of work."""
    x = torch.zeros((8192, 8192), dtype=torch.bfloat16, device="cuda")

    def busy():
        for _ in range(40):
            x.mul_(0) @ x
    busy()  # (the products' own setting up)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    return s, busy


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_trees(kind, late):
    from block_sparse_long_index_gb300 import MsaTreeDecode
    from test_gpu_tree import Case
    stream, busy = late
    c = Case(kind, [50, 3], 5, 8, 2, 64, 16, seed=1)
    want = [t.clone() for t in c.run()]
    ctx, par = i32(c.ctx), i32(c.parents)
    torch.cuda.synchronize()
    busy()
    dec = MsaTreeDecode(c.pool, c.B, c.T, c.table.shape[1], c.H_q)
    out, lse = dec(c.q, c.table, ctx, par, None, c.scale, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kind", ["bf16", "kv4"])
def test_pools_and_tables(kind, late):
    from block_sparse_long_index_gb300 import Kv4Pool, KvPool, PagedCache
    stream, busy = late
    k, v, cu, zero, n = rows(40, 2, 64, seed=2), rows(40, 2, 64, seed=3), i32([0, 40]), i32([0]), i32([40])

    def fill(stream):
        pool = (KvPool if kind == "bf16" else Kv4Pool).empty(6, 16, 2, 64)
        cache = PagedCache.empty(1, 4, 6, 16, pool.tensors())
        cache.reserve(zero, n, stream=stream)
        pool.append(k, v, cu, zero, cache.page_table, stream=stream)
        return pool.tensors() + [cache.page_table, cache.ctx_len, cache.refs]

    want = fill(None)
    torch.cuda.synchronize()
    busy()
    got = fill(stream)
    torch.cuda.synchronize()
    assert int(want[-2][0]) == 40
    for a, b in zip(got, want):
        assert torch.equal(a, b)
