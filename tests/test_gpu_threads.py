"""Calls of two host threads at once, each with an object, tensors and a stream of its own."""
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
    """One and two query tiles need different amounts of shared memory of one kernel."""
    from test_gpu_tree import Case
    cases = [Case("bf16", [50, 3], T, 8, 2, d, 16, seed=T) for T in (2, 40)]
    want = [[t.clone() for t in c.run()] for c in cases]
    runs = []
    for c in cases:
        ctx, par, s = i32(c.ctx), i32(c.parents), torch.cuda.Stream()
        runs.append(lambda c=c, ctx=ctx, par=par, s=s: c.dec(c.q, c.table, ctx, par, None, c.scale, stream=s))
    torch.cuda.synchronize()
    at_once(*runs)
    for c, w in zip(cases, want):
        assert torch.equal(c.dec.out, w[0]) and torch.equal(c.dec.lse, w[1])
