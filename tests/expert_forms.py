"""Cases that between them reach every product kernel of csrc/expert.hip, with
inputs on which the kernels are exact: small integers whose sums stay below 2^24
in fp32, gates past 17.4 where 1 + exp(-g) is 1, and h below 2^16.  An output is
then the bf16 rounding of the exact value, to the bit.

A kernel is named by the parameters that tell them apart:
  ("thin", kind, out, waves), ("wide", kind, out, weight tiles, row tiles),
  ("down", kind, weight tiles)
with kinds bf16, stream (bf16 with non-temporal reads), fp4, int4g32, int4g64,
int4g128 and outs gated, bf16, f32."""

import ctypes
import os
import subprocess

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_ep_send_amd", "csrc")
KINDS = {"bf16": ("bf16", 0), "stream": ("bf16", 0), "fp4": ("fp4", 32), "int4g32": ("int4", 32),
         "int4g64": ("int4", 64), "int4g128": ("int4", 128)}
OUTS = ("gated", "bf16", "f32")          # the values 0, 1, 2 of FewOut

# R, E, N, K of row calls
ROWS = {
    "small": [(3, 2, 72, 256), (3, 2, 72, 4224), (9, 3, 72, 256), (40, 2, 72, 256),
              (100, 16, 1032, 256), (320, 16, 1032, 256), (100, 3, 72, 256)],
    # matrices of 64 MB and more
    "stream": [(3, 64, 264, 2048), (3, 64, 72, 8192), (9, 1024, 80, 448), (40, 2, 1032, 16384),
               (100, 16, 4104, 512), (320, 16, 4104, 512), (100, 3, 1032, 10944)],
}
# T, K, E, H, I of layers
LAYERS = {
    "small": [(3, 2, 4, 256, 128), (3, 2, 4, 4224, 128), (9, 2, 4, 6272, 128), (9, 8, 8, 256, 256),
              (20, 8, 8, 256, 256), (16, 8, 16, 1152, 256), (40, 8, 16, 1152, 256),
              (40, 8, 8, 256, 256), (3, 2, 4, 256, 1536), (2, 1, 2, 128, 4224)],
    "stream": [(3, 2, 32, 2048, 512), (3, 2, 32, 4096, 256), (9, 8, 8, 1024, 4096),
               (20, 8, 8, 1024, 4096), (16, 8, 16, 2048, 1024), (40, 8, 16, 2048, 1024),
               (40, 8, 8, 2048, 2048), (3, 2, 16, 1024, 2048), (3, 2, 8, 1024, 4096)],
}


def cases():
    """(call, kind, sizes) of every case.  Plain bf16 gets channels that end
    inside a 128-channel block."""
    for kind in KINDS:
        size = "stream" if kind == "stream" else "small"
        for R, E, N, K in ROWS[size]:
            yield "rows", kind, (R, E, N, K + (8 if kind == "bf16" else 0))
        for T, K, E, H, I in LAYERS[size]:
            more = 8 if kind == "bf16" else 0
            yield "layer", kind, (T, K, E, H + more, I + more)


# ---------------------------------------------------------------------------
# which kernels a case takes, by the library's own rules
# ---------------------------------------------------------------------------

RULES = r"""
#include "expert_rules.h"
using namespace epdc;
extern "C" void form(int slots, int rows, int per_token, int experts, int N, int K, int out,
                     int bf16, int* f) {
  const FewForm v = few_form(FewSizes{slots, rows, per_token, experts, N, K}, FewOut(out), bf16);
  f[0] = v.waves, f[1] = v.weight_tiles, f[2] = v.row_tiles;
}
extern "C" int streams(int experts, int rows, int K) {
  return streams_bf16(reinterpret_cast<const void*>(4096), experts, rows, K);
}
extern "C" int joined(int slots, int hidden, int inner) {
  return few_down_joined(slots, hidden, inner);
}
extern "C" int tiles(int hidden, int bf16) { return down_tiles(hidden, bf16); }
"""


def rules(folder):
    src, out = os.path.join(folder, "rules.cpp"), os.path.join(folder, "rules.so")
    with open(src, "w") as f:
        f.write(RULES)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-I", CSRC, "-o", out,
                    src], check=True)
    return ctypes.CDLL(out)


def _product(lib, kind, out, slots, rows, per_token, experts, N, K):
    f = (ctypes.c_int * 3)()
    lib.form(slots, rows, per_token, experts, N, K, OUTS.index(out), KINDS[kind][0] == "bf16", f)
    return ("thin", kind, out, f[0]) if f[0] else ("wide", kind, out, f[1], f[2])


def _kind(lib, kind, experts, rows, K):
    if KINDS[kind][0] != "bf16":
        return kind
    return "stream" if lib.streams(experts, rows, K) else "bf16"


def kernels(lib, call, kind, sizes):
    if call == "rows":
        R, E, N, K = sizes
        return [_product(lib, _kind(lib, kind, E, N, K), "bf16", R, R, 1, E, N, K)]
    T, K, E, H, I = sizes
    first = _product(lib, _kind(lib, kind, E, 2 * I, H), "gated", T * K, T, 1, E, I, H)
    k2 = _kind(lib, kind, E, H, I)
    if lib.joined(T * K, H, I):
        return [first, ("down", k2, lib.tiles(H, KINDS[kind][0] == "bf16"))]
    return [first, _product(lib, k2, "f32", T * K, T * K, K, E, H, I)]


def every_kernel():
    for kind in KINDS:
        for out in OUTS:
            yield from (("thin", kind, out, w) for w in (4, 8))
            yield from (("wide", kind, out, 2, m) for m in (1, 2, 3))
            if out != "gated":
                yield from (("wide", kind, out, 1, m) for m in (1, 2))
        yield "down", kind, 1
        if KINDS[kind][0] != "bf16":
            yield "down", kind, 2


# ---------------------------------------------------------------------------
# inputs and exact outputs
# ---------------------------------------------------------------------------

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float32)


def weights(rng, kind, E, N, K, small=False):
    """(tensors as the package takes them, values [E, N, K] float32) of integer
    matrices.  small: codes of magnitudes up to 3."""
    fmt, group = KINDS[kind]
    if fmt == "bf16":
        v = rng.integers(-3, 4, (E, N, K)).astype(np.float32) if small else \
            rng.integers(-8, 9, (E, N, K)).astype(np.float32)
        return [torch.from_numpy(v).to(torch.bfloat16), None], v
    code = rng.integers(0, 16, (E, N, K), dtype=np.uint8)
    if small:
        code = rng.integers(0, 4, (E, N, K), dtype=np.uint8)
        code = code + 6 if fmt == "int4" else code | rng.integers(0, 2, (E, N, K), dtype=np.uint8) << 3
    return _w4(rng, fmt, group, code)


def _w4(rng, fmt, group, code):
    E, N, K = code.shape
    # most groups have scale 1 (fp4: 2), some twice that
    up = (rng.integers(0, 3, (E, N, K // group)) == 0).astype(np.uint8)
    factor = np.repeat(np.float32(1) + up, group, -1)
    if fmt == "int4":
        v = (code.astype(np.float32) - 8) * factor
        scale = torch.from_numpy(1.0 + up).to(torch.bfloat16)
    else:
        m = 2 * E2M1[code & 7]
        v = np.where(code > 7, -m, m) * factor
        scale = torch.from_numpy(up + np.uint8(128))
    q = code[..., 0::2] | code[..., 1::2] << 4
    return [torch.from_numpy(q), scale], v


def rows_inputs(kind, sizes):
    R, E, N, K = sizes
    rng = np.random.default_rng([R, E, N, K])
    t, v = weights(rng, kind, E, N, K)
    x = rng.integers(-4, 5, (R, K)).astype(np.float32)
    # half of the rows to one expert, some to none, the rest anywhere
    ids = np.where(rng.random(R) < 0.5, E - 1, rng.integers(0, E, R)).astype(np.int32)
    if R > 3:
        ids[1], ids[R - 2] = -1, E
    return t, v, torch.from_numpy(x).to(torch.bfloat16), torch.from_numpy(ids)


def rows_exact(v, x, ids):
    """float64 on x's device; v [E, N, K] on the host."""
    y = torch.zeros(x.shape[0], v.shape[1], dtype=torch.float64, device=x.device)
    for e in range(v.shape[0]):
        r = (ids == e).nonzero()[:, 0]
        if r.numel():
            w = torch.from_numpy(v[e]).to(x.device).double()
            y[r] = x[r].double() @ w.t()
            assert float((x[r].double().abs() @ w.abs().t()).max()) < 2 ** 24
    return y


SURE = 16                                # channels of x that are 1 and make every gate large


def layer_inputs(kind, sizes):
    """The gate of every row is some 100 to 200 by its first SURE channels, the
    up value comes from up to 64 other channels of +-1."""
    T, K, E, H, I = sizes
    rng = np.random.default_rng([T, K, E, H, I])
    fmt, group = KINDS[kind]
    sure = rng.permutation(H)[:SURE]
    if fmt == "bf16":
        _, v13 = weights(rng, kind, E, 2 * I, H, small=True)
        v13[:, :I, sure], v13[:, I:, sure] = 8, 0
        t13 = [torch.from_numpy(v13).to(torch.bfloat16), None]
    else:
        (q, _), _ = weights(rng, kind, E, 2 * I, H, small=True)
        q = q.numpy()
        code = np.stack([q & 15, q >> 4], -1).reshape(E, 2 * I, H)
        code[:, :I, sure], code[:, I:, sure] = (15, 8) if fmt == "int4" else (5, 0)
        t13, v13 = _w4(rng, fmt, group, code)
    t2, v2 = weights(rng, kind, E, H, I)
    x = np.zeros((T, H), np.float32)
    others = np.setdiff1d(np.arange(H), sure)
    for t in range(T):
        at = rng.choice(others, min(64, len(others)), replace=False)
        x[t, at] = rng.choice([-1, 1], len(at))
    x[:, sure] = 1
    idx = np.argsort(rng.random((T, max(E, K))), 1)[:, :K].astype(np.int64) % E
    idx[rng.random((T, K)) < 0.1] = -1
    idx[:, 0] = np.where(rng.random(T) < 0.3, E - 1, idx[:, 0])        # an expert with more rows
    w = rng.choice([1.0, 2.0], (T, K)).astype(np.float32)
    return t13, v13, t2, v2, torch.from_numpy(x).to(torch.bfloat16), torch.from_numpy(idx), \
        torch.from_numpy(w)


def layer_exact(v13, v2, x, idx, w):
    I = v2.shape[2]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    size = torch.zeros_like(out)
    for e in range(v2.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        w13 = torch.from_numpy(v13[e]).to(x.device).double()
        gu = x[t].double() @ w13.t()
        g, u = gu[:, :I], gu[:, I:]
        assert float(g.min()) > 17.4
        h = g * u
        assert float(h.abs().max()) < 2 ** 16
        w2 = torch.from_numpy(v2[e]).to(x.device).double()
        y = h @ w2.t()
        out.index_add_(0, t, y * w[t, k].double()[:, None])
        size.index_add_(0, t, y.abs() * w[t, k].double()[:, None])
        # a slot's sum, in parts and in any order: terms of random signs, whose partial
        # sums stay within eight times the 2-norm of all
        norm = ((h ** 2) @ (w2 ** 2).t()).sqrt()
        assert float(norm.max()) * 8 < 2 ** 24
    assert float(size.max()) < 2 ** 24
    return out
