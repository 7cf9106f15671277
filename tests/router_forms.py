"""Plain 64-bit forms of the calls before the dispatch on the CPU, with bounds on
how far a kernel that sums in fp32 may be from them.

Unit roundoffs: a rounding to bf16 2^-8 relative, to e4m3 2^-4, to fp32 2^-24; an
addition on the matrix cores 2^-23 (they may truncate).  A term of a sum passes
through so many additions at most as its bound counts."""

import numpy as np
import torch

BF16, E4M3, F32, STEP = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24, 2.0 ** -23
TINY = 2.0 ** -133          # smallest bf16 magnitude
SMALL = 2.0 ** -149         # smallest fp32 magnitude


def f64(t):
    return t.detach().cpu().double().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


# ---- norm ---------------------------------------------------------------------

# additions a square passes through: 64 in a thread, 6 over a wave, 16 over the
# waves; its own rounding, the quotient, eps, the root (halved) and the reciprocal
NORM_SUM = (64 + 6 + 16 + 4) * F32


def norm_ref(s, w, eps):
    """(rstd, its bound, y, its bound in fp32) of rows s [T, H]."""
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    y = s * rstd[:, None] * w
    e = NORM_SUM / 2 + 3 * F32
    return rstd, rstd * e, y, np.abs(y) * (e + 3 * F32) + SMALL


def norm_backward_ref(dy, s, w, rstd, dres=None):
    """(dx, bound, dw, bound): the row's sum as in the forward; the weight's
    gradient over up to T / 256 + 2 rows a workgroup, 64 partial rows a thread and
    16 threads."""
    T, H = s.shape
    n, g = s * rstd[:, None], dy * w
    mean, mag = (g * n).mean(1), np.abs(g * n).mean(1)
    dx = rstd[:, None] * (g - n * mean[:, None])
    e = (64 + 6 + 16 + 6) * F32 * mag[:, None]
    tol = rstd[:, None] * (4 * F32 * np.abs(g) + np.abs(n) * (e + 4 * F32 * np.abs(mean[:, None])))
    if dres is not None:
        dx = dx + dres
        tol = tol + 2 * F32 * (np.abs(dx) + np.abs(dres))
    dw = (dy * n).sum(0)
    dtol = (T / 256 + 2 + 64 + 16 + 4) * F32 * np.abs(dy * n).sum(0) + SMALL
    return dx, tol + BF16 * np.abs(dx) + TINY, dw, dtol


# ---- router -------------------------------------------------------------------

def logits_ref(x, w):
    """(logits, bound): a product passes through 32 additions in its instruction,
    one for each later instruction, wave and split."""
    H = x.shape[1]
    return x @ w.T, (H / 32 + 32 + 4 + 256) * STEP * (np.abs(x) @ np.abs(w).T) + SMALL


# sizes with several turns of every product's ring of stages, the last turn not whole,
# and several workgroups of experts: by logits_shape 64 tokens by 64, 128 and 256
# experts, 16 and 32 tokens by 256, 128 by 128 in the wide form; by dx_shape 64, 32 and
# 16 tokens.  tests/test_router_rules.py holds them to that.
DEEP = [(8195, 64, 1032), (8200, 128, 648), (2000, 256, 4872), (2047, 300, 1672), (1000, 700, 1096),
        (17, 1024, 65536), (16, 1024, 16392), (9001, 129, 648), (8195, 300, 648), (2100, 1000, 456),
        (4099, 513, 840), (2048, 400, 1032)]


def logits_backward_ref(dl, x, w):
    T, E = dl.shape
    dx, dw = dl @ w, dl.T @ x
    dx_tol = (2.0 ** -16 + (2 * E / 32 + 36 + 4) * STEP) * (np.abs(dl) @ np.abs(w))
    dw_tol = (F32 + (3 * T / 32 + 32 + 64) * STEP) * (np.abs(dl).T @ np.abs(x))
    return dx, dx_tol + BF16 * np.abs(dx) + TINY, dw, dw_tol + SMALL


# ---- choice -------------------------------------------------------------------

def scores64(l, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))),
                            np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        e = np.exp(l - np.fmax.reduce(l, axis=1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def route_ref(l, K, score="softmax", bias=None, groups=1, kept=1, top=2, renorm=True, scale=1.0,
              count=None):
    """(idx, weights) token by token, as the header words it."""
    T, E = l.shape
    idx, w = np.full((T, K), -1, np.int64), np.zeros((T, K))
    s = scores64(l, score)
    if kept == groups:
        groups = kept = 1
    by_score = bias is not None or (groups > 1 and top == 2)
    key = s + (0 if bias is None else bias) if by_score else l
    for t in range(T if count is None else min(T, max(0, count))):
        ok = [e for e in range(E) if l[t, e] > -np.inf and key[t, e] > -np.inf]
        if groups > 1:
            size, worth = E // groups, {}
            for e in ok:
                worth.setdefault(e // size, []).append(key[t, e])
            worth = {g: sum(sorted(v, reverse=True)[:top]) for g, v in worth.items()}
            stay = sorted(worth, key=lambda g: (-worth[g], g))[:kept]
            ok = [e for e in ok if e // size in stay]
        pick = sorted(ok, key=lambda e: (-key[t, e], e))[:K]
        if not pick:
            continue
        idx[t, :len(pick)] = pick
        with np.errstate(all="ignore"):
            if renorm and score == "softmax":
                p = np.exp(l[t, pick] - max(l[t, pick]))
            else:
                p = s[t, pick]
            total = p.sum() if renorm else 1.0
            w[t, :len(pick)] = scale * p / total if total != 0 else 0.0
    return idx, w


def route_backward_ref(dw, l, idx, score="softmax", renorm=True, scale=1.0):
    """By the chain rule from the definition, slot by slot.  The second result
    bounds what 64 bits leave: sizes that cancel count in full."""
    T, E = l.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    s = scores64(l, score)
    for t in range(T):
        ks = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E]
        if not ks:
            continue
        e, d = idx[t, ks], scale * dw[t, ks]
        with np.errstate(all="ignore"):
            if score == "softmax" and renorm:
                q = np.exp(l[t, e] - max(l[t, e]))
                q = q / q.sum()
                g, m = q * (d - (d * q).sum()), q * (np.abs(d) + np.abs(d * q).sum())
                np.add.at(out[t], e, g)
                np.add.at(size[t], e, m)
                continue
            p = s[t, e]
            total = p.sum() if renorm else 1.0
            if total == 0:
                continue
            ds = (d - ((d * p).sum() / total if renorm else 0.0)) / total
            dm = (np.abs(d) + (np.abs(d * p).sum() / total if renorm else 0.0)) / total
            if score == "sigmoid":
                x = np.exp(-np.abs(l[t, e]))
                np.add.at(out[t], e, ds * x / (1 + x) ** 2)
                np.add.at(size[t], e, dm * x / (1 + x) ** 2)
            else:
                np.add.at(out[t], e, ds * p)
                np.add.at(size[t], e, dm * p)
                out[t] -= s[t] * (ds * p).sum()
                size[t] += s[t] * (dm * p).sum()
    return out, F32 * np.abs(out) + 2.0 ** -44 * size + SMALL


# ---- quantized rows --------------------------------------------------------------

def permute_ref(rows, token_row, out):
    out = out.copy()
    for t in range(token_row.shape[0]):
        for r in token_row[t]:
            if 0 <= r < out.shape[0]:
                out[r] = rows[t]
    return out


def check(got, ref, tol, what=""):
    """Every element within its bound; prints the worst before it fails."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), (what, "not finite", np.argwhere(~np.isfinite(got))[:5])
    ratio = np.abs(got - ref) / np.maximum(tol, np.finfo(np.float64).tiny)
    if ratio.size:
        at = np.unravel_index(np.argmax(ratio), ratio.shape)
        assert ratio[at] <= 1, (what, at, got[at], ref[at], tol[at])
