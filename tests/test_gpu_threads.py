"""Calls of two host threads at once, each with an object, tensors and a stream of its own."""
import ctypes
import threading

import pytest
import torch

from test_gpu_kv4 import i32

pytestmark = pytest.mark.gpu


def at_once(*calls, times=2000):
    """Runs each call `times` times in a thread of its own, all threads at once."""
    go, failed = threading.Barrier(len(calls)), []

    def loop(call):
        try:
            go.wait()
            for _ in range(times):
                call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("d", [64, 128])
def test_trees_of_few_and_of_many_rows(d):
    """One and two query tiles need different amounts of shared memory of one kernel.  (Calls of the C function itself: Python
    threads run side by side within it alone.)"""
    from block_sparse_long_index_gb300 import msa
    from test_gpu_tree import Case
    cases = [Case("bf16", [50, 3], T, 8, 2, d, 16, seed=T) for T in (2, 40)]
    want = [[t.clone() for t in c.run()] for c in cases]
    runs = []
    for c in cases:
        at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        s, ctx, par, w = torch.cuda.Stream(), i32(c.ctx), i32(c.parents), c.dec.workspace
        a = (at(c.q), ctypes.byref(c.pool.c), at(c.table), c.table.shape[1], at(ctx), None, at(par), c.B, c.T, c.H_q, c.scale, at(c.dec.out),
             at(c.dec.lse), at(w), w.numel(), ctypes.c_void_p(s.cuda_stream))
        keep = (ctx, par)

        def run(f=msa.raw().msa_tree_decode_paged, a=a, s=s, keep=keep):
            for _ in range(200):
                if f(*a):
                    raise RuntimeError("a launch failed")
            s.synchronize()

        runs.append(run)
    torch.cuda.synchronize()
    at_once(*runs, times=150)
    for c, w in zip(cases, want):
        assert torch.equal(c.dec.out, w[0]) and torch.equal(c.dec.lse, w[1])


def serving_calls():
    """A call of each kind whose first CUDA call may be the encoding of a tensor map."""
    from block_sparse_long_index_gb300 import MsaDecodeKv4, MsaDensePrefill, MsaPrefill
    from test_gpu_rope import rows
    from test_gpu_tree import Case
    out = {}
    for kind, T in (("bf16", 3), ("kv4", 3), ("kv4", 40)):
        c = Case(kind, [50, 3], T, 8, 2, 64, 16, seed=T)
        c.run()
        a = (c.q, c.table, i32(c.ctx), i32(c.parents), None, c.scale)
        out["tree %s %d" % (kind, T)] = lambda c=c, a=a: c.dec(*a)
        if kind == "kv4" and T == 3:
            one, q = MsaDecodeKv4(c.pool, 2, c.table.shape[1], 8), rows(2, 8, 64, seed=1)
            ctx = i32(c.ctx)
            out["dense decode"] = lambda c=c, one=one, q=q, ctx=ctx: one.dense(q, c.table, ctx)
    pre, x = MsaPrefill(300, 4, 2, 64, 32, 64, 3), [rows(300, *y, seed=2) for y in ((4, 64), (2, 64), (2, 64), (2, 32), (32,))]
    out["prefill"] = lambda: pre(*x)
    dense, cu = MsaDensePrefill(300, 4, 2, 64, 2), i32([0, 100, 300])
    out["dense prefill"] = lambda: dense(*x[:3], cu)
    return out


@pytest.mark.parametrize("name", ["tree bf16 3", "tree kv4 3", "tree kv4 40", "dense decode", "prefill", "dense prefill"])
def test_the_first_cuda_call_of_a_thread(name):
    call = serving_calls()[name]
    torch.cuda.synchronize()
    at_once(call, times=1)


def test_decode_steps_of_small_and_of_large_tables():
    """The scan keeps a maximum for each block that a table has room for."""
    from block_sparse_long_index_gb300 import Kv4Pool, MsaDecodeKv4
    from test_gpu_rope import rows
    pool, idx = Kv4Pool.empty(4, 128, 2, 64), rows(4, 128, 64, seed=1)
    x, y = rows(512, 2, 64, seed=2), rows(512, 2, 64, seed=3)
    pool.store(x, y, i32([0, 512]), i32([0]), i32([[0, 1, 2, 3]]))
    runs, want = [], []
    for B, max_pages in ((2, 4), (310, 8192)):
        run, s = MsaDecodeKv4(pool, B, max_pages, 4, d_I=64, Bk=64, k=4), torch.cuda.Stream()
        table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        table[:, :4] = i32([0, 1, 2, 3])
        a = (rows(B, 4, 64, seed=4), rows(B, 2, 64, seed=5), idx, table, i32([400] * B))
        want.append([t.clone() for t in run(*a)[:2]])
        runs.append((run, a, s))
    torch.cuda.synchronize()
    at_once(*[lambda run=run, a=a, s=s: run(*a, stream=s) for run, a, s in runs], times=1000)
    for (run, *_), w in zip(runs, want):
        assert torch.equal(run.out, w[0]) and torch.equal(run.lse, w[1])


def test_prefills_of_different_lengths():
    """The inversion counts in shared memory what each block of keys is chosen by; the combine holds a position's partials."""
    from block_sparse_long_index_gb300 import MsaPrefill
    from test_gpu_rope import rows
    runs, want = [], []
    for N, H_q, k in ((300, 2, 3), (70000, 8, 16)):
        run, s = MsaPrefill(N, H_q, 1, 64, 32, 64, k), torch.cuda.Stream()
        a = [rows(N, *x, seed=6 + i) for i, x in enumerate(((H_q, 64), (1, 64), (1, 64), (1, 32), (32,)))]
        want.append([t.clone() for t in run(*a)])
        runs.append((run, a, s))
    torch.cuda.synchronize()
    at_once(*[lambda run=run, a=a, s=s: run(*a, stream=s) for run, a, s in runs], times=200)
    for (run, *_), w in zip(runs, want):
        assert torch.equal(run.block_idx, w[2])
