"""The serving classes together: what their calls return stays until its own buffer is written again, the MSA step after
a cache was forked, freed and compacted, page calls that refuse, and two prefills at once."""
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
