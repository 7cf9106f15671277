"""Plain 64-bit forms of the expert-side operators on the CPU, with bounds on
how far a kernel that sums in fp32 may be from them, and seeded inputs.

Unit roundoffs: fp32 2^-24; a chain of n fp32 additions is off by at most
n * 2^-23 of the sum of magnitudes (2^-23 a step: the matrix cores may truncate
where an addition would round); rounding to bf16 by half a step, 2^-8 relative."""

import numpy as np
import torch

BF16 = 2.0 ** -8
STEP = 2.0 ** -23
TINY = 2.0 ** -133          # smallest bf16 magnitude

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])

FORMATS = [("bf16", 0), ("int4", 32), ("int4", 64), ("int4", 128), ("fp4", 32)]


def bf16(a):
    """numpy array -> bf16 tensor (CPU), rounded to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


def f64(t):
    return t.double().numpy()


def make_weights(rng, fmt, group, E, N, K):
    """(tensors as the package takes them, on the CPU; values; magnitudes that
    bound the partial sums) of E matrices [N, K]."""
    if fmt == "bf16":
        q = bf16(rng.standard_normal((E, N, K)) / np.sqrt(K))
        v = f64(q)
        return (q, None), v, np.abs(v)
    q = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "int4":
        s = bf16(rng.uniform(0.5, 1.5, (E, N, K // group)) / (4.6 * np.sqrt(K)))
        sv = f64(s)
    else:
        e = 127 + int(np.round(np.log2(1 / (2.7 * np.sqrt(K)))))
        s = torch.from_numpy(rng.integers(e - 1, e + 2, (E, N, K // group)).astype(np.uint8))
        sv = None
    v = w4_values(q, s.numpy() if fmt == "fp4" else sv, fmt, group)
    # int4 sums (16 + c) x and 24 x apart: up to 31 + 24 steps a channel
    mag = np.abs(v) if fmt == "fp4" else 55.0 * np.repeat(sv, group, -1)
    return (torch.from_numpy(q), s), v, mag


def w4_values(q, scale, fmt, group):
    c = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    if fmt == "int4":
        return (c.astype(np.float64) - 8) * np.repeat(scale.astype(np.float64), group, -1)
    s = np.ldexp(1.0, np.repeat(scale.astype(np.int64), group, -1) - 127)
    s = np.where(np.repeat(scale, group, -1) == 255, np.nan, s)
    return E2M1[c] * s


def matvec_ref(x, ids, v, mag):
    """(y, bound) [R, N]; rows with an id outside [0, E) are NaN."""
    R, K = x.shape
    y = np.full((R, v.shape[1]), np.nan)
    tol = np.zeros_like(y)
    for r in range(R):
        if 0 <= ids[r] < v.shape[0]:
            y[r] = v[ids[r]] @ x[r]
            tol[r] = BF16 * np.abs(y[r]) + 1.01 * K * STEP * (mag[ids[r]] @ np.abs(x[r])) + TINY
    return y, tol


def silu64(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def moe_ref(x, idx, w, v13, m13, v2, m2, first, biases=()):
    """(out, bound) [T, H].  h is carried in two bf16 parts, the first cut and
    the rest rounded: off by at most 2^-7 * 2^-8 of its size."""
    T, H = x.shape
    E, _, I = v2.shape
    K = idx.shape[1]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        size = np.zeros(H)
        for k in range(K):
            e = int(idx[t, k]) - first
            if idx[t, k] < 0 or not 0 <= e < E:
                continue
            gu = v13[e] @ x[t]
            err = H * STEP * (m13[e] @ np.abs(x[t]))
            g, u, eg, eu = gu[:I], gu[I:], err[:I], err[I:]
            h = silu64(g) * u
            # |silu'| <= 1.1; the exponential and the quotient: (|g| + 8) 2^-22 relative
            d = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu64(g)) * eu + \
                np.abs(h) * ((np.abs(g) + 8) * 2.0 ** -22 + 2.0 ** -15) + 2 * TINY
            y = v2[e] @ h
            wk = float(w[t, k])
            out[t] += wk * y
            # two products a channel
            tol[t] += abs(wk) * (np.abs(v2[e]) @ d + 2.02 * I * STEP * (m2[e] @ (np.abs(h) + d)))
            size += abs(wk) * np.abs(y)
        for b in biases:
            out[t] += b[t]
            size += np.abs(b[t])
        tol[t] += (K + 4) * STEP * size
    return out, tol * (1 + BF16) + BF16 * np.abs(out) + TINY


def check(got, ref, tol, what=""):
    """Every element within its bound; prints the worst before it fails."""
    got = got.detach().cpu().double().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), (what, "not finite", np.argwhere(~np.isfinite(got))[:5])
    ratio = np.abs(got - ref) / np.maximum(tol, np.finfo(np.float64).tiny)
    if ratio.size:
        at = np.unravel_index(np.argmax(ratio), ratio.shape)
        assert ratio[at] <= 1, (what, at, got[at], ref[at], tol[at])


def topk(rng, T, K, E, unrouted=0.0):
    idx = np.argsort(rng.random((T, max(E, K))), axis=1)[:, :K].astype(np.int64)
    idx[idx >= E] = -1
    idx[rng.random((T, K)) < unrouted] = -1
    w = rng.random((T, K)).astype(np.float32)
    return idx, w / w.sum(1, keepdims=True)
