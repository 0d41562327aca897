"""msa_dense_prefill_varlen on the GPU against a 64-bit implementation."""
import math

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

CASES = [
    # lens, H_q, H_kv, d
    ([1], 1, 1, 64),
    ([1], 8, 1, 128),
    ([2, 1, 1, 3], 4, 2, 128),
    ([0, 5, 0, 0, 17, 0], 8, 8, 64),
    ([128], 8, 1, 128),
    ([129], 8, 1, 128),
    ([127, 128, 129, 1], 16, 2, 128),
    ([32, 33, 31, 64, 65], 24, 3, 128),
    ([300, 41], 8, 4, 64),
    ([257, 255], 2, 2, 128),
    ([600], 4, 4, 64),
    ([1000, 3, 514], 32, 8, 128),
    ([777], 12, 3, 128),
]


def make(lens, H_q, H_kv, d, pad=0, seed=0, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N = sum(lens) + pad
    mk = lambda h: torch.randn(N, h, d, generator=g, device="cuda").mul(spread).to(torch.bfloat16)  # noqa: E731
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return mk(H_q), mk(H_kv), mk(H_kv), cu


def run(q, k, v, cu, scale, stream=None):
    from block_sparse_long_index_gb300 import MsaDensePrefill
    plan = MsaDensePrefill(q.shape[0], q.shape[1], k.shape[1], q.shape[2], cu.numel() - 1)
    plan.out.fill_(7.0)
    plan.lse.fill_(7.0)
    out, lse = plan(q, k, v, cu, scale, stream=stream)
    return plan, out, lse


@pytest.mark.parametrize("lens,H_q,H_kv,d", CASES)
def test_against_64_bits(lens, H_q, H_kv, d):
    q, k, v, cu = make(lens, H_q, H_kv, d)
    scale = 1 / math.sqrt(d)
    plan, out, lse = run(q, k, v, cu, scale)
    assert plan.device_status() == 0
    ref.check_attention(out, lse.T, *ref.dense_prefill(q, k, v, lens, scale), d, max(lens))


@pytest.mark.parametrize("H_q,H_kv,d", [(8, 1, 128), (4, 2, 64), (3, 3, 128)])
def test_large_scores(H_q, H_kv, d):
    """Scores of several hundred, a rising maximum from tile to tile."""
    lens = [513, 130]
    q, k, v, cu = make(lens, H_q, H_kv, d, spread=4.0)
    k *= torch.linspace(0.2, 3.0, k.shape[0], device="cuda")[:, None, None].to(torch.bfloat16)
    plan, out, lse = run(q, k, v, cu, 0.25)
    assert plan.device_status() == 0
    ref.check_attention(out, lse.T, *ref.dense_prefill(q, k, v, lens, 0.25), d, max(lens))


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H_q,H_kv,d", [(8, 1, 128), (2, 2, 64)])
def test_rows_of_no_sequence(fill, H_q, H_kv, d):
    """Rows behind the last sequence hold anything, are not read into results and stay as they were."""
    lens = [70, 200, 5]
    n = sum(lens)
    q, k, v, cu = make(lens, H_q, H_kv, d, pad=90)
    for t in (q, k, v):
        t[n:] = fill
    plan, out, lse = run(q, k, v, cu, 0.1)
    assert plan.device_status() == 0
    assert bool((out[n:] == 7.0).all()) and bool((lse[:, n:] == 7.0).all())
    r = ref.dense_prefill(q[:n], k[:n], v[:n], lens, 0.1)
    ref.check_attention(out[:n], lse[:, :n].T, *r, d, max(lens))


def test_all_sequences_empty():
    q, k, v, _ = make([40], 4, 2, 64)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    plan, out, lse = run(q, k, v, cu, 0.1)
    assert plan.device_status() == 0
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


@pytest.mark.parametrize("cu", [[1, 40], [0, 30, 20, 40], [0, 41], [0, -3, 40]])
def test_bad_offsets(cu):
    from block_sparse_long_index_gb300 import msa
    q, k, v, _ = make([40], 4, 2, 64)
    plan, out, lse = run(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 0.1)
    assert plan.device_status() == msa.MSA_ERR_BAD_INDEX
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_equal_to_warmup_forward():
    """One prompt is the dense branch of warmup mode: the same definition, another kernel."""
    from block_sparse_long_index_gb300 import msa
    N, H_q, H_kv, d = 700, 16, 2, 128
    q, k, v, cu = make([N], H_q, H_kv, d)
    qi = torch.randn(N, H_kv, 128, device="cuda").to(torch.bfloat16)
    ki = torch.randn(N, 128, device="cuda").to(torch.bfloat16)
    o2, l2 = torch.empty_like(q), torch.empty(H_q, N, device="cuda")
    li = torch.empty(H_kv, N, device="cuda")
    msa.msa_warmup_fwd(q, k, v, qi, ki, msa.shape(N, H_q, H_kv, d, 128, 64, 1), 0.1, o2, l2, li)
    _, out, lse = run(q, k, v, cu, 0.1)
    assert float((out.float() - o2.float()).norm() / o2.float().norm()) < 2 * ref.BF16_HALF
    assert float((lse - l2).abs().max()) < 1e-4


def test_stream_and_graph():
    lens = [333, 64, 1]
    q, k, v, cu = make(lens, 8, 2, 128)
    from block_sparse_long_index_gb300 import MsaDensePrefill
    plan = MsaDensePrefill(q.shape[0], 8, 2, 128, 3)
    want = plan(q, k, v, cu, 0.1)[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.out.zero_()
    torch.cuda.synchronize()
    plan(q, k, v, cu, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(plan.out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan(q, k, v, cu, 0.1)
    q2, k2, v2, _ = make(lens, 8, 2, 128, seed=5)
    q.copy_(q2), k.copy_(k2), v.copy_(v2)
    cu.copy_(torch.tensor([0, 100, 250, 398], dtype=torch.int32))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    ref.check_attention(plan.out, plan.lse.T, *ref.dense_prefill(q, k, v, [100, 150, 148], 0.1), 128, 150)


def test_two_calls_at_once():
    """Two plans on two streams; and the same inputs give the same bits."""
    a, b = make([900, 50], 8, 1, 128, seed=1), make([20, 700], 8, 8, 64, seed=2)
    wa, wb = run(*a, 0.1)[1].clone(), run(*b, 0.1)[1].clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        oa, ob = run(*a, 0.1, stream=s1)[1], run(*b, 0.1, stream=s2)[1]
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


@pytest.mark.parametrize("H_q,H_kv,d", [(8, 1, 128), (4, 1, 64), (2, 2, 128), (1, 1, 64)])
@pytest.mark.parametrize("at", [0, 5, 130, 300])
def test_values_that_are_not_finite(at, H_q, H_kv, d):
    """A NaN or an infinity in V (and a NaN in K) reaches the rows that see it, and no row before it."""
    lens = [310, 40]
    q, k, v, cu = make(lens, H_q, H_kv, d)
    want = run(q, k, v, cu, 0.1)[1].clone()
    v[at, 0, 3] = math.nan
    v[at, 0, 5] = math.inf
    v[at + 4, 0, 5] = -math.inf
    plan, out, _ = run(q, k, v, cu, 0.1)
    assert plan.device_status() == 0
    gs = H_q // H_kv
    o, w = out[:, :gs], want[:, :gs]
    clean = [c for c in range(d) if c not in (3, 5)]
    assert torch.equal(o[:, :, clean], w[:, :, clean]) and torch.equal(out[:, gs:], want[:, gs:])
    assert torch.equal(o[:at], w[:at]) and torch.equal(o[310:], w[310:])
    assert bool(torch.isnan(o[at:310, :, 3]).all())
    assert bool((o[at:at + 4, :, 5] == math.inf).all()) and bool(torch.isnan(o[at + 4:310, :, 5]).all())
    q, k, v, cu = make(lens, H_q, H_kv, d)
    k[at, 0, 7] = math.nan
    _, out, lse = run(q, k, v, cu, 0.1)
    assert torch.equal(out[:at], want[:at]) and torch.equal(out[310:], want[310:])
    assert bool(torch.isnan(out[at:310, :gs]).all()) and bool(torch.isnan(lse[:gs, at:310]).all())
