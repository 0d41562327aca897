"""Plain 64-bit implementations of the serving operators (dense attention, the 4-bit cache format, page tables),
written from their definitions for the tests; they share no code with the library."""
import math

import numpy as np
import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2  # half a step, relative to the value


# ---------------------------------------------------------------- attention
def attend(q, k, v, scale):
    """q [h, d], k, v [n, d] float64: (out [h, d], lse [h], A [h, d] = sum_j p_j |v_j|, S [h] = largest
    scale sum_c |q_c k_c|)."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    x = (q @ k.T) * scale
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    return p @ v, lse, p @ v.abs(), (q.abs() @ k.abs().T).amax(1) * scale


def dense_prefill(q, k, v, lens, scale):
    """Packed causal attention in 64 bits: out [N, H_q, d], lse [N, H_q], A and S as attend's."""
    N, H_q, d = q.shape
    gs = H_q // k.shape[1]
    out = torch.zeros(N, H_q, d, dtype=torch.float64, device=q.device)
    lse = torch.zeros(N, H_q, dtype=torch.float64, device=q.device)
    A, S = torch.zeros_like(out), torch.zeros_like(lse)
    q, k, v = q.double(), k.double(), v.double()
    a = 0
    for n in lens:
        if n == 0:
            continue
        unseen = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
        for h in range(H_q):
            g = h // gs
            kk, vv = k[a:a + n, g], v[a:a + n, g]
            x = (q[a:a + n, h] @ kk.T * scale).masked_fill(unseen, -math.inf)
            ls = torch.logsumexp(x, 1)
            p = torch.exp(x - ls[:, None])
            out[a:a + n, h], lse[a:a + n, h], A[a:a + n, h] = p @ vv, ls, p @ vv.abs()
            S[a:a + n, h] = (q[a:a + n, h].abs() @ kk.abs().T).masked_fill(unseen, 0).amax(1) * scale
        a += n
    return out, lse, A, S


def check_attention(out, lse, ref, ref_lse, A, S, d, n):
    """out (bf16, [..., h, d]) and lse (fp32, [..., h]) against the 64-bit results.

    The score of a pair is an fp32 sum of d exact products: off by at most d 2^-24 sum |q k| scale (S is the
    largest such sum), twice that for the running maximum's share, and 2^-22 for the exponential: eps.
    Probabilities are rounded to bf16 (half a step) before they meet V, the result once more; fp32 sums over n
    terms and the row sum add n 2^-24, taken pairwise within tiles: 2^-24 (n / 64 + 64) covers them."""
    eps = 2 * d * 2.0 ** -24 * S + 2.0 ** -21
    acc = 2.0 ** -24 * (n / 64 + 64)
    tol = BF16_HALF * ref.abs() + (BF16_HALF * (1 + BF16_HALF) + 2 * eps[..., None] + 2 * acc) * A + 1e-30
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), "out: worst %.3f of the tolerance" % float((err / tol).max())
    ltol = eps + acc + 2.0 ** -22 * ref_lse.abs().clamp(max=1e30) + 2.0 ** -22
    fin = torch.isfinite(ref_lse)
    assert bool((torch.isfinite(lse) == fin).all()) and bool((lse[~fin].double() == ref_lse[~fin]).all())
    lerr = (lse.double() - ref_lse).abs()[fin]
    assert bool((lerr <= ltol[fin]).all()), "lse: worst %.3f of the tolerance" % float((lerr / ltol[fin]).max())


# ---------------------------------------------------------------- 4-bit format (numpy, 64 bits)
def scale_values():
    b = np.arange(255)
    return 2.0 ** (b // 8 - 20) * (1 + b % 8 / 8)


def quantize(x):
    """x [..., d] float64: (codes [..., d] 0..15, scale bytes [..., 4]) by the definition."""
    g = x.reshape(*x.shape[:-1], 4, -1)
    sv = scale_values()
    codes = np.full(g.shape, 8, np.int64)
    scales = np.full(g.shape[:-1], 255, np.int64)
    for i in np.ndindex(*g.shape[:-1]):
        row = g[i]
        if not np.isfinite(row).all():
            continue
        ok = np.nonzero(7 * sv >= np.abs(row).max())[0]
        s = ok[0] if len(ok) else 254
        scales[i] = s
        codes[i] = 8 + np.clip(np.rint(row / sv[s]), -7, 7).astype(np.int64)  # rint: ties to even
    return codes.reshape(x.shape), scales


def values(codes, scales):
    """codes [..., d] 0..15 and scale bytes [..., 4] -> float64."""
    sv = np.append(scale_values(), np.nan)[scales]
    g = codes.reshape(*codes.shape[:-1], 4, -1)
    return ((g - 8) * sv[..., None]).reshape(codes.shape)


def pack(codes):
    """codes [..., d] -> bytes [..., d / 2]: nibble n of a word of 8 is channel 2n, or 2(n - 4) + 1 from n = 4 on."""
    w = codes.reshape(*codes.shape[:-1], -1, 8)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    nib = w[..., order]
    return (nib[..., 0::2] | nib[..., 1::2] << 4).astype(np.uint8).reshape(*codes.shape[:-1], -1)


def unpack(packed):
    b = packed.astype(np.int64).reshape(*packed.shape[:-1], -1, 4)
    nib = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 8)
    order = [0, 2, 4, 6, 1, 3, 5, 7]
    out = np.empty_like(nib)
    out[..., order] = nib
    return out.reshape(*packed.shape[:-1], -1)


# ---------------------------------------------------------------- pages (plain Python lists)
class PagesRef:
    """Page tables by their definition: lists of page ids, a count per page, page contents as one number each."""

    def __init__(self, n_seqs, max_pages, n_pages, page):
        self.page, self.max_pages = page, max_pages
        self.table = [[] for _ in range(n_seqs)]
        self.ctx, self.refs = [0] * n_seqs, [0] * n_pages
        self.data = list(range(n_pages))  # a page's content

    def _free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, seqs, lens):
        need = [-(-n // self.page) - len(self.table[s]) for s, n in zip(seqs, lens)]
        free = self._free()
        if sum(need) > len(free):
            return False
        for s, n, c in zip(seqs, lens, need):
            ids, free = free[:c], free[c:]
            self.table[s] += ids
            for i in ids:
                self.refs[i] = 1
            self.ctx[s] = n
        return True

    def fork(self, src, dst):
        free = self._free()
        if sum(self.ctx[s] % self.page > 0 for s in src) > len(free):
            return False
        lens = [self.ctx[s] for s in src]
        rows = [list(self.table[s]) for s in src]
        for row, n, d in zip(rows, lens, dst):
            full = n // self.page
            new = row[:full]
            for i in new:
                self.refs[i] += 1
            if n % self.page:
                last, free = free[0], free[1:]
                self.data[last] = self.data[row[full]]
                self.refs[last] = 1
                new.append(last)
            self.table[d], self.ctx[d] = new, n
        return True

    def free(self, seqs):
        for s in seqs:
            for i in self.table[s]:
                self.refs[i] -= 1
            self.table[s], self.ctx[s] = [], 0

    def compact(self):
        live = [i for i, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [i for i in range(n) if self.refs[i] == 0]
        to = {i: i for i in live if i < n}
        for a, b in zip([i for i in live if i >= n], holes):
            to[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.data[b] = self.data[a]
        self.table = [[to[i] for i in row] for row in self.table]
        return [to.get(i, -1) for i in range(len(self.refs))], n
