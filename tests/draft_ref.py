"""Plain 64-bit implementations of the operators of a speculative decode step (rotary positions, attention of drafted trees,
their verification, the accepted branch), written from their definitions for the tests; they share no code with the library."""
import math

import numpy as np
import torch


# ---------------------------------------------------------------- rotary positions
def turn(x, positions, freqs, interleaved=False, amplitude=1.0, inverse=False):
    """x [N, H, d] float64 with the first 2 len(freqs) channels turned by positions (integers) times freqs (radians).
    Angles are reduced modulo a turn in 128-bit integers, so that they are right at any position."""
    n = len(freqs)
    two_pi = 0x3243F6A8885A308D313198A2E03707344 * 2  # 2 pi 2^128
    ang = np.empty((len(positions), n))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            a, b = float(f).as_integer_ratio()
            num = (int(p) * a << 128) // b % two_pi  # p f modulo 2 pi, in 2^-128
            ang[i, j] = num / 2.0 ** 128
    c = torch.tensor(np.cos(ang), device=x.device)[:, None] * amplitude
    s = torch.tensor(np.sin(ang), device=x.device)[:, None] * (-amplitude if inverse else amplitude)
    y = x.clone()
    ai = torch.arange(n, device=x.device) * 2 if interleaved else torch.arange(n, device=x.device)
    bi = ai + (1 if interleaved else n)
    y[..., ai] = x[..., ai] * c - x[..., bi] * s
    y[..., bi] = x[..., bi] * c + x[..., ai] * s
    return y


def turn_error(x, freqs, positions, interleaved=False, amplitude=1.0):
    """What fp32 arithmetic may be off by, for every channel of turned rows: cos and sin by 2^-24 and half a step of the table
    (|p| 2^-65 turns), times the amplitude (rounded: 2^-24); each product and their sum by 2^-24."""
    n = len(freqs)
    ai = torch.arange(n, device=x.device) * 2 if interleaved else torch.arange(n, device=x.device)
    bi = ai + (1 if interleaved else n)
    p = torch.as_tensor(np.abs(np.asarray(positions, np.float64)), device=x.device)[:, None, None]
    e = torch.zeros_like(x)
    pair = x[..., ai].abs() + x[..., bi].abs()
    e[..., ai] = e[..., bi] = abs(amplitude) * pair * (4 * 2.0 ** -24 * (1 + 2.0 ** -20) + p * 2.0 ** -65 * 2 * math.pi)
    return e


# ---------------------------------------------------------------- drafted trees
def ancestors(parents):
    """For each node, itself and the nodes above it."""
    out = []
    for i in range(len(parents)):
        line, j = [], i
        while j >= 0:
            line.append(j)
            j = parents[j]
        out.append(line)
    return out


def tree_attend(q, k, v, ctx, parents, scale):
    """q [T, H_q, d], k and v [ctx + T, H_kv, d] float64 of one sequence: out, lse, and the quantities that tolerances need
    (A = sum p |v|, S = the largest scale sum |q k|), each [T, H_q, ...]."""
    T, H_q, d = q.shape
    gs = H_q // k.shape[1]
    out, A = torch.zeros_like(q), torch.zeros_like(q)
    lse, S = torch.zeros(T, H_q, dtype=torch.float64, device=q.device), torch.zeros(T, H_q, dtype=torch.float64, device=q.device)
    for i, line in enumerate(ancestors(parents)):
        at = torch.tensor(list(range(ctx)) + [ctx + j for j in line], device=q.device)
        for h in range(H_q):
            kk, vv = k[at, h // gs], v[at, h // gs]
            x = kk @ q[i, h] * scale
            lse[i, h] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[i, h]) if lse[i, h] > -math.inf else torch.zeros_like(x)
            out[i, h], A[i, h], S[i, h] = p @ vv, p @ vv.abs(), (kk.abs() @ q[i, h].abs()).max() * scale
    return out, lse, A, S


def tree_of(rng, T, kind):
    """Parents of T nodes: "chain", "wide" (all below node 0), "roots" (all roots), or random."""
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "wide":
        return [-1] + [0] * (T - 1)
    if kind == "roots":
        return [-1] * T
    return [-1] + [int(rng.integers(max(0, j - 5), j)) for j in range(1, T)]


# ---------------------------------------------------------------- verification
def verify(p, q, tokens, parents, u, u_last):
    """One sequence, by the rule's own steps: p [T, V], q [T, V] or None, float64 of the fp32 values.  (path, next token, how
    near the nearest comparison was, relative to what it compares: with sums held to 2^-48, a case nearer than 2^-40 has
    no one answer and is no test.)"""
    T, V = p.shape
    node, path, near = 0, [0], math.inf
    r = p[0].copy()
    W = 1.0
    j = 1
    while j < T:
        if parents[j] == node:
            x = tokens[j]
            # r / W is what is left of the target's distribution
            lhs, rhs = (q[node, x] if q is not None else 1.0) * float(u[j]) * W, r[x]
            near = min(near, abs(lhs - rhs) / max(lhs, rhs, 1e-300))
            if lhs < rhs:
                path.append(j)
                node, r, W = j, p[j].copy(), 1.0
            elif q is not None:
                r = np.maximum(0.0, r - W * q[node])
                W = math.fsum(r)
            else:
                W -= r[x]
                r[x] = 0.0
        j += 1
    if not r.sum() > 0:
        r = p[node]
    cum = np.cumsum(r.astype(np.longdouble))
    target = np.longdouble(float(u_last)) * cum[-1]
    near = min(near, float(np.min(np.abs(cum - target)) / cum[-1]))
    return path, int(np.searchsorted(cum, target, side="right")), near


# ---------------------------------------------------------------- the accepted branch
def accept(rows, base, path):
    """rows: a sequence's token contents, a list; what is left of it."""
    return rows[:base] + [rows[base + j] for j in path]
