"""Verification of drafted trees where the outcome hangs on the last bits of sums over long vocabularies: tokens drawn and drafts
accepted next to a border, against sums of integers.  Probabilities from 2^-35 on and their differences are exact in the
library's units of 2^-58, each smaller one is off by 2^-59 at most, and u times a sum is worked out in 64-bit floating point
(2^-52); the cases here are 2^-40 or more from their border, and hold far fewer than 2^19 tokens below 2^-35 in anything that is
summed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** 61
SURE = 0.99999988  # a random number that rejects every draft with p well below q


def rows_of(B, V, seed, spread=3.0):
    """[B, V] fp32 distributions, and others near them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    p, q = (torch.empty((B, V), device="cuda") for _ in range(2))
    for b in range(B):
        x = torch.randn(V, generator=g, device="cuda") * spread
        p[b] = torch.softmax(x, 0)
        q[b] = torch.softmax(x + 0.7 * torch.randn(V, generator=g, device="cuda"), 0)
    return p, q


def total(r):
    """The sum of float64 values (multiples of a unit, to half of it), in any order the same."""
    return float((r * UNIT).round().long().sum()) / UNIT


def near_border(r, lo=2.0 ** -40, hi=2.0 ** -38):
    """A u_last next to a border of the cumulative sum of r (float64 [V]), between lo and hi of the sum away from it, and the
    token that it draws."""
    cum = torch.cumsum((r * UNIT).round().long(), 0)
    c = cum.double() / float(cum[-1])
    u = c.float()
    off = (u.double() - c).abs()
    some = ((off >= lo) & (off <= hi) & (u < 1.0)).nonzero().flatten()
    for i in some[(c[some] - 0.6).abs().argsort()[:9]].tolist():  # (where most of the sum's errors have come together)
        if float((c - u[i].double()).abs().min()) >= lo:  # (no other border is nearer)
            return float(u[i]), int((c > u[i].double()).nonzero()[0])
    raise AssertionError("no such border")


def verify(p, q, tokens, parents, u, ul):
    """p, q [B, T, V] on the GPU, the others as lists."""
    from block_sparse_long_index_gb300 import DraftVerifier
    B, T, V = p.shape
    i32, f32 = (lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")), (lambda x: torch.tensor(x, dtype=torch.float32, device="cuda"))
    run = DraftVerifier(B, T, V)
    path, n, nxt = run(p, i32(tokens), i32(parents), f32(u), f32(ul), q)
    assert run.device_status() == 0
    return path.tolist(), n.tolist(), nxt.tolist()


def reject(p, q, times):
    """Drafts that the rule rejects one after the other (with u = SURE), and what is left of p (float64 [V])."""
    r, W, tokens = p.double(), 1.0, []
    for _ in range(times):
        x = int((q.double() * W - r).argmax())
        assert float(q[x]) * SURE * W > float(r[x]) * (1 + 2.0 ** -20)
        tokens.append(x)
        r = (r - W * q.double()).clamp(min=0.0)
        W = total(r)
    return tokens, r, W


@pytest.mark.parametrize("rejections", [0, 1, 2])
@pytest.mark.parametrize("B,V", [(3, 128000), (20, 128000), (40, 128000), (2, (1 << 20) + 3), (20, 1 << 20), (40, (1 << 20) + 1)])
def test_draws_next_to_a_border(B, V, rejections):
    p, q = rows_of(B, V, V + B + rejections)
    T = 1 + rejections
    told = [reject(p[b], q[b], rejections) for b in range(B)]
    ul, want = zip(*[near_border(r) for _, r, _ in told])
    wide = [x[:, None].expand(B, T, V).contiguous() for x in (p, q)]
    path, n, nxt = verify(*wide, [[0] + t for t, _, _ in told], [[-1] + [0] * rejections] * B, [[SURE] * T] * B, list(ul))
    assert n == [1] * B
    assert nxt == list(want)


@pytest.mark.parametrize("B", [2, 40])
def test_draws_without_certain_drafts_next_to_a_border(B):
    V = (1 << 20) + 2
    p, _ = rows_of(B, V, 5 + B)
    tokens = [[int(x) for x in p[b].topk(3).indices[1:]] for b in range(B)]
    ul, want = [], []
    for b in range(B):
        r = p[b].double()
        r[tokens[b]] = 0.0
        u, token = near_border(r)
        ul.append(u)
        want.append(token)
    path, n, nxt = verify(p[:, None].expand(B, 3, V).contiguous(), None, [[0] + t for t in tokens], [[-1, 0, 0]] * B, [[SURE] * 3] * B, ul)
    assert n == [1] * B and nxt == want


@pytest.mark.parametrize("B", [1, 40])
def test_draws_from_16_million_tokens(B):
    """Every token is about as likely as the others: a sum off by 2^-24 of itself draws another one."""
    V = (1 << 24) + 5
    g = torch.Generator(device="cuda").manual_seed(6)
    p = torch.empty((B, 1, V), device="cuda")
    ul, want = [], []
    for b in range(B):
        p[b, 0] = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
        cum = torch.cumsum((p[b, 0].double() * UNIT).round().long(), 0)
        c = cum.double() / float(cum[-1])
        u = (torch.rand(64, generator=g, device="cuda") * 0.9).tolist()
        ul.append(next(x for x in u if float((c - x).abs().min()) > 2.0 ** -32))
        want.append(int(torch.searchsorted(c, torch.tensor([ul[-1]], device="cuda", dtype=torch.float64), right=True)))
    path, n, nxt = verify(p, None, [[0]] * B, [[-1]] * B, [[0.5]] * B, ul)
    assert nxt == want


@pytest.mark.parametrize("B,V", [(3, 128000), (20, 1 << 20), (40, (1 << 20) + 1)])
def test_drafts_accepted_next_to_the_border(B, V):
    """The second draft of a node is accepted where u q W < r, W the sum that the first one's rejection left."""
    p, q = rows_of(B, V, 7 + B)
    tokens, us, want = [], [], []
    for b in range(B):
        first, r, W = reject(p[b], q[b], 1)
        qw = q[b].double() * W
        u = (r / qw).float()
        off = (u.double() * qw - r) / r
        fits = (r > 0) & (u < 1.0) & (off.abs() >= 2.0 ** -39) & (off.abs() <= 2.0 ** -37)
        x = int(fits.nonzero().flatten()[0])
        tokens.append([0] + first + [x])
        us.append([SURE, SURE, float(u[x])])
        want.append(2 if float(off[x]) < 0 else 1)
    wide = [x[:, None].expand(B, 3, V).contiguous() for x in (p, q)]
    path, n, nxt = verify(*wide, tokens, [[-1, 0, 0]] * B, us, [0.5] * B)
    assert len(set(want)) == 2 or B < 8
    assert n == want and [x[1] for x in path] == [2 if w == 2 else -1 for w in want]


def test_the_outcome_does_not_hang_on_the_batch():
    """One tree with 40 random numbers as near to a border as fp32 has them: alone, in a batch of 20 and of 40."""
    V = (1 << 19) + 3
    p, q = rows_of(1, V, 9)
    tokens, r, _ = reject(p[0], q[0], 1)
    c = torch.cumsum(r, 0) / r.sum()
    near = (c.float().double() - c).abs() + (c.float() >= 1.0)
    ul = c.float()[near.argsort()[:40]].tolist()
    got = {}
    for B in (1, 20, 40):
        wide = [x[:, None].expand(B, 2, V).contiguous() for x in (p, q)]
        got[B] = sum((verify(*wide, [[0] + tokens] * B, [[-1, 0]] * B, [[SURE] * 2] * B, ul[i:i + B])[2] for i in range(0, 40, B)), [])
    assert got[1] == got[20] == got[40]


def test_rows_that_are_no_distributions():
    """Values above 1 and sums far above it: the walk ends, and a token that has a share is drawn."""
    B, V = 3, 70001
    p = torch.zeros((B, 1, V), device="cuda")
    p[0, 0, ::7] = 0.5
    p[1, 0, 11], p[1, 0, 5000] = 3e38, 1.0
    p[2, 0] = 1.0
    path, n, nxt = verify(p, None, [[0]] * B, [[-1]] * B, [[0.5]] * B, [0.999] * B)
    assert n == [1] * B and all(float(p[b, 0, nxt[b]]) > 0 for b in range(B))
