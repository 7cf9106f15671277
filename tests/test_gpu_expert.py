"""Few-row expert products, the layer for a few tokens and the 4-bit quantizer
against plain 64-bit forms (tests/expert_helpers.py derives the bounds)."""

import numpy as np
import pytest
import torch

from tests.expert_helpers import (E2M1, FORMATS, bf16, check, f64, make_weights, matvec_ref,
                                  moe_ref, topk, w4_values)
from tests.gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

import combine_ep_send_amd as ep  # noqa: E402

DEV = "cuda:0"


def dev_weights(t, fmt, group):
    q, s = t
    return q.to(DEV) if fmt == "bf16" else ep.W4Weights(q.to(DEV), s.to(DEV), fmt, group)


# (rows, experts, N, K): one of everything; odd tiles; row counts around the
# 16- and 32-row tiles; K around the 128-channel block (bf16 also between)
SHAPES = [(1, 1, 8, 128), (1, 1, 64, 1024), (2, 1, 136, 2176), (4, 3, 40, 640), (3, 2, 24, 256), (16, 1, 72, 384), (17, 1, 40, 128),
          (33, 3, 16, 640), (70, 2, 136, 256), (5, 40, 48, 128), (200, 7, 56, 256)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("R,E,N,K", SHAPES)
def test_matvec(fmt, group, R, E, N, K):
    rng = np.random.default_rng(R * 1000 + N)
    t, v, mag = make_weights(rng, fmt, group, E, N, K)
    x = bf16(rng.standard_normal((R, K)))
    ids = rng.integers(0, E, R).astype(np.int32)
    ref, tol = matvec_ref(f64(x), ids, v, mag)
    w = dev_weights(t, fmt, group)
    y = ep.ep_expert_matvec(x.to(DEV), w, torch.from_numpy(ids).to(DEV))
    check(y, ref, tol, "ids")
    if E == 1:
        y1 = ep.ep_expert_matvec(x.to(DEV), w)
        assert torch.equal(y.view(torch.int16), y1.view(torch.int16))


@pytest.mark.parametrize("K", [8, 24, 32, 40, 120, 136, 520, 1000])
def test_matvec_bf16_channel_tails(K):
    rng = np.random.default_rng(K)
    t, v, mag = make_weights(rng, "bf16", 0, 2, 40, K)
    # what lies behind a row must not be multiplied in: the next row is not finite
    for R in (4, 5):
        x = bf16(rng.standard_normal((R, K)))
        x[2] = float("inf")
        ids = np.array([0, 1, 1, 0, 1], np.int32)[:R]
        y = ep.ep_expert_matvec(x.to(DEV), t[0].to(DEV), torch.from_numpy(ids).to(DEV))
        keep = [r for r in range(R) if r != 2]
        ref, tol = matvec_ref(f64(x)[keep], ids[keep], v, mag)
        check(y[keep], ref, tol)


@pytest.mark.parametrize("R", [3, 21])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_rows_without_an_expert_get_zeros(fmt, group, R):
    rng = np.random.default_rng(5)
    E, N, K = 3, 40, 256
    t, v, mag = make_weights(rng, fmt, group, E, N, K)
    x = bf16(rng.standard_normal((R, K)))
    ids = rng.integers(0, E, R).astype(np.int32)
    out = [1, 2] if R == 3 else [2, 3, 11, 20]
    ids[out] = [-1, E, -2 ** 31, 2 ** 31 - 1][:len(out)]
    x[out] = float("nan")
    buf = torch.full((R + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = ep.ep_expert_matvec(x.to(DEV), dev_weights(t, fmt, group), torch.from_numpy(ids).to(DEV),
                            out=buf[:R])
    assert (buf[R:] == 7).all() and (buf[out].view(torch.int16) == 0).all()
    ref, tol = matvec_ref(f64(x), ids, v, mag)
    keep = [r for r in range(R) if r not in out]
    check(y[keep], ref[keep], tol[keep])
    none = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    z = ep.ep_expert_matvec(x.to(DEV), dev_weights(t, fmt, group), none, out=buf[1:R + 1])
    assert (z.view(torch.int16) == 0).all() and (buf[R + 1:] == 7).all()


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_a_matrix_that_is_not_finite_stays_with_its_rows(fmt, group):
    rng = np.random.default_rng(6)
    E, N, K, R = 3, 24, 128, 6
    t, v, mag = make_weights(rng, fmt, group, E, N, K)
    if fmt == "bf16":
        t[0][1] = float("nan")
    elif fmt == "int4":
        t[1][1] = float("inf")
    else:
        t[1][1] = 255
    x = bf16(rng.standard_normal((R, K)))
    ids = np.array([0, 1, 2, 0, 2, 1], np.int32)
    y = ep.ep_expert_matvec(x.to(DEV), dev_weights(t, fmt, group), torch.from_numpy(ids).to(DEV))
    ref, tol = matvec_ref(f64(x), ids, v, mag)
    keep = [0, 2, 3, 4]
    check(y[keep], ref[keep], tol[keep])
    assert not torch.isfinite(y[[1, 5]]).any()


def test_1024_rows_and_1024_experts():
    rng = np.random.default_rng(7)
    t, v, mag = make_weights(rng, "int4", 128, 1024, 8, 128)
    x = bf16(rng.standard_normal((1024, 128)))
    w = dev_weights(t, "int4", 128)
    for ids in (rng.permutation(1024), np.full(1024, 1023), rng.integers(0, 1024, 1024)):
        ids = ids.astype(np.int32)
        ref, tol = matvec_ref(f64(x), ids, v, mag)
        check(ep.ep_expert_matvec(x.to(DEV), w, torch.from_numpy(ids).to(DEV)), ref, tol)


def test_fp4_extreme_scales():
    """Scale bytes 0 (2^-127), 1 and 254: the products are exact powers of two
    times e2m1 values, so one channel at a time is exact.  With byte 254 the
    codes of 2 and more stand for 2^128 and more, past bf16 and fp32 alike:
    infinities, by the format's definition in the header."""
    K = 128
    q = np.zeros((1, 16, K // 2), np.uint8)
    q[0, :, 0] = np.arange(16)                 # row n: code n in channel 0
    x = torch.zeros(3, K, dtype=torch.bfloat16)
    x[0, 0], x[1, 0], x[2, 0] = 1.0, 2.0 ** 100, 2.0 ** -20
    for byte, rows in ((0, (1,)), (1, (1,)), (127, (0, 1, 2)), (254, (2,))):
        s = torch.full((1, 16, K // 32), byte, dtype=torch.uint8)
        y = ep.ep_expert_matvec(x.to(DEV), ep.W4Weights(torch.from_numpy(q).to(DEV), s.to(DEV),
                                                        "fp4", 32))
        for r in rows:
            with np.errstate(over="ignore"):
                w = (E2M1 * 2.0 ** (byte - 127)).astype(np.float32).astype(np.float64)
            want = w * float(x[r, 0])
            assert np.array_equal(f64(y[r].cpu()), want + 0.0), (byte, r)


def test_int4_activations_up_to_their_limit():
    K = 256
    rng = np.random.default_rng(8)
    t, v, mag = make_weights(rng, "int4", 64, 1, 24, K)
    x = bf16(rng.standard_normal((2, K)))
    x[0] *= 2.0 ** 118                          # below 2^122 in magnitude
    x[1] *= 2.0 ** -100
    ids = np.zeros(2, np.int32)
    ref, tol = matvec_ref(f64(x), ids, v, mag)
    check(ep.ep_expert_matvec(x.to(DEV), dev_weights(t, "int4", 64)), ref, tol)


# ---------------------------------------------------------------------------
# layer
# ---------------------------------------------------------------------------

LAYERS = [  # T, K, E here, experts in all, first, H, I
    (1, 1, 1, 1, 0, 128, 128), (1, 8, 32, 32, 0, 256, 128), (3, 2, 8, 8, 0, 512, 256),
    (4, 16, 40, 64, 7, 384, 640), (2, 3, 4, 4, 0, 1152, 128), (5, 3, 4, 64, 20, 256, 384), (17, 2, 3, 3, 0, 128, 640), (64, 16, 20, 40, 10, 128, 128),
    (128, 8, 16, 16, 0, 256, 128), (40, 1, 1, 2, 1, 384, 256)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,K,E,all_e,first,H,I", LAYERS)
def test_layer(fmt, group, T, K, E, all_e, first, H, I):
    rng = np.random.default_rng(T * 100 + K)
    t13, v13, m13 = make_weights(rng, fmt, group, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, fmt, group, E, H, I)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, all_e, unrouted=0.1 if T > 4 else 0.0)
    out = ep.ep_moe_tokens(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV),
                           dev_weights(t13, fmt, group), dev_weights(t2, fmt, group), first)
    ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, first)
    check(out, ref, tol)


@pytest.mark.parametrize("H,I", [(8, 8), (40, 24), (136, 200), (264, 1000)])
def test_layer_bf16_tails_biases_and_mixed_formats(H, I):
    rng = np.random.default_rng(H)
    T, K, E = 7, 2, 3
    t13, v13, m13 = make_weights(rng, "bf16", 0, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, "bf16", 0, E, H, I)
    x, b = bf16(rng.standard_normal((T, H))), [bf16(rng.standard_normal((T, H))) for _ in "ab"]
    idx, w = topk(rng, T, K, E, unrouted=0.3)
    idx[4] = -1                                # a token with no expert: the biases alone
    args = [torch.from_numpy(a).to(DEV) for a in (idx, w)]
    for n in (0, 1, 2):
        bias = [t.to(DEV) for t in b[:n]]
        out = ep.ep_moe_tokens(x.to(DEV), *args, t13[0].to(DEV), t2[0].to(DEV),
                               bias=(bias if n == 2 else bias[0] if n else None))
        ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 0, [f64(t) for t in b[:n]])
        check(out, ref, tol, n)
        if n == 0:
            assert (out[4].view(torch.int16) == 0).all()
    if H % 128 == 8 and I % 8 == 0:            # one matrix bf16, the other 4-bit
        I2 = 256
        t13, v13, m13 = make_weights(rng, "bf16", 0, E, 2 * I2, H)
        t2, v2, m2 = make_weights(rng, "int4", 64, E, H, I2)
        out = ep.ep_moe_tokens(x.to(DEV), *args, t13[0].to(DEV), dev_weights(t2, "int4", 64))
        ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 0)
        check(out, ref, tol, "mixed")


@pytest.mark.parametrize("T", [4, 64])
def test_layer_ids_of_every_kind(T):
    """Ids far outside, one expert named by every slot (more rows than one
    tile of any variant), the same expert twice in a token, nothing routed."""
    rng = np.random.default_rng(11)
    K, E, H, I = 16, 4, 128, 128
    t13, v13, m13 = make_weights(rng, "fp4", 32, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, "fp4", 32, E, H, I)
    x = bf16(rng.standard_normal((T, H)))
    w = rng.random((T, K)).astype(np.float32)
    odd = np.full((T, K), 2 ** 62, np.int64)
    odd[::2] = -2 ** 63
    odd[1, 3], odd[2, 15], odd[-1, 0] = 1000, 1003, 1004
    twice = rng.integers(1000, 1000 + E, (T, K)).astype(np.int64)
    twice[:, 1] = twice[:, 0]
    for name, idx in (("odd", odd), ("one", np.full((T, K), 1002, np.int64)), ("twice", twice),
                      ("none", np.full((T, K), -1, np.int64))):
        out = ep.ep_moe_tokens(x.to(DEV), torch.from_numpy(idx).to(DEV),
                               torch.from_numpy(w).to(DEV), dev_weights(t13, "fp4", 32),
                               dev_weights(t2, "fp4", 32), 1000)
        ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 1000)
        check(out, ref, tol, name)


def test_layer_skips_what_it_does_not_name():
    """NaN in the weights of unrouted slots, in the rows of tokens that are not
    routed here and in the matrices of experts nobody names reaches nothing."""
    rng = np.random.default_rng(12)
    T, K, E, H, I = 9, 3, 6, 128, 128
    t13, v13, m13 = make_weights(rng, "bf16", 0, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, "bf16", 0, E, H, I)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, 4)
    idx[5] = -1
    idx[2, 1] = -1
    w[5], w[2, 1] = np.nan, np.inf
    x[5] = float("nan")
    t13[0][4:], t2[0][4:] = float("nan"), float("inf")
    out = ep.ep_moe_tokens(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV),
                           t13[0].to(DEV), t2[0].to(DEV))
    xs = f64(x)
    xs[5] = 0
    ref, tol = moe_ref(xs, idx, np.nan_to_num(w, nan=0, posinf=0), v13, m13, v2, m2, 0)
    check(out, ref, tol)


@pytest.mark.parametrize("tokens", [3, 9, 50, 128])
def test_layer_gives_the_same_bits_again_and_keeps_to_its_buffers(tokens):
    rng = np.random.default_rng(13)
    T, K, E, H, I = tokens, 8, 16, 256, 256
    t13, _, _ = make_weights(rng, "int4", 128, E, 2 * I, H)
    t2, _, _ = make_weights(rng, "int4", 128, E, H, I)
    x = bf16(rng.standard_normal((T, H))).to(DEV)
    idx, w = (torch.from_numpy(a).to(DEV) for a in topk(rng, T, K, E))
    w13, w2 = dev_weights(t13, "int4", 128), dev_weights(t2, "int4", 128)
    n = ep.ep_moe_tokens_workspace_bytes(T, K, H, I)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=DEV)
    first = ep.ep_moe_tokens(x, idx, w, w13, w2, out=buf[1:T + 1], workspace=ws[:n]).clone()
    assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (ws[n:] == 0xA5).all()
    for fill in (0, 0xFF):
        ws.fill_(fill)
        again = ep.ep_moe_tokens(x, idx, w, w13, w2, workspace=ws[:n])
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,K,E,H,I", [(4, 16, 64, 6272, 128), (8, 8, 9, 6272, 128),
                                       (16, 4, 2, 2176, 128), (13, 5, 3, 2176, 128),
                                       (4, 8, 9, 2176, 384), (11, 3, 9, 2176, 384)])
def test_layer_of_up_to_64_slots_and_many_channels(fmt, group, T, K, E, H, I):
    """The sum joined to the products at its most slots and widest tiles, and
    one slot past it."""
    rng = np.random.default_rng(T + K)
    t13, v13, m13 = make_weights(rng, fmt, group, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, fmt, group, E, H, I)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, E)
    out = ep.ep_moe_tokens(x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV),
                           dev_weights(t13, fmt, group), dev_weights(t2, fmt, group))
    ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 0)
    check(out, ref, tol)


@pytest.mark.parametrize("R", [2, 5, 40])
def test_matrices_near_the_size_limit(R):
    """Five matrices of 2^31 - 2^18 bytes (over 10 GB): offsets inside a matrix
    reach the 31st bit, those of the later ones pass the 32nd."""
    N, K = 16384, 65528
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.zeros(5, N, K, dtype=torch.bfloat16, device=DEV)
    rows = [0, 1, 8191, 8192, N - 17, N - 1]
    w[:, rows] = torch.randn(5, len(rows), K, device=DEV, generator=g).to(torch.bfloat16)
    x = torch.randn(R, K, device=DEV, generator=g).to(torch.bfloat16)
    ids = torch.tensor([4, 1, 4, 0, 3] * 8, dtype=torch.int32, device=DEV)[:R]
    y = ep.ep_expert_matvec(x, w, ids)
    picked = f64(w[:, rows].cpu())
    ref, tol = matvec_ref(f64(x.cpu()), ids.cpu().numpy(), picked, np.abs(picked))
    check(y[:, rows], ref, tol)
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert (y[:, rest] == 0).all()


def test_empty_calls():
    w13 = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros(2, 8, 8, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(0, 8, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(0, 2, dtype=torch.int64, device=DEV)
    w = torch.zeros(0, 2, device=DEV)
    assert ep.ep_moe_tokens(x, idx, w, w13, w2).shape == (0, 8)
    assert ep.ep_expert_matvec(x, w2[:1]).shape == (0, 8)
    q = ep.ep_quantize_w4(torch.zeros(0, 128, dtype=torch.bfloat16, device=DEV))
    assert q.q.shape == (0, 64) and q.scale.shape == (0, 1)


# ---------------------------------------------------------------------------
# quantizer
# ---------------------------------------------------------------------------

def quantize_ref(v, fmt, group):
    """Codes and scales by definition; v float32 [.., K]."""
    g = v.reshape(*v.shape[:-1], -1, group)
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    amax = np.where(bad, np.float32(1), amax).astype(np.float32)
    g = np.where(bad[..., None], np.float32(0), g)
    if fmt == "int4":
        s = torch.from_numpy(amax / np.float32(7)).to(torch.bfloat16).float().numpy()
        d = np.where(s == 0, np.float32(1), s)[..., None]
        q = np.clip(np.rint(g / d), -8, 7)
        q = np.where(s[..., None] == 0, 0, q).astype(np.int64) + 8
        scale = np.where(bad, np.nan, s)
    else:
        a = (amax / np.float32(6)).astype(np.float64)
        e = np.where(a > 0, np.ceil(np.log2(np.where(a > 0, a, 1.0))), 0).astype(np.int64)
        e = np.where(np.ldexp(1.0, e - 1) >= a, e - 1, e)        # log2 may land one off
        e = np.where(np.ldexp(1.0, e) < a, e + 1, e)
        byte = np.where(amax == 0, 0, np.maximum(e + 127, 0))
        r = np.abs(g.astype(np.float64)) * np.ldexp(1.0, 127 - byte)[..., None]
        grid = E2M1[:8]
        dist = np.abs(r[..., None] - grid)
        q = 7 - np.argmin(dist[..., ::-1], -1)                   # of two nearest the upper ...
        low = np.argmin(dist, -1)
        q = np.where((low != q) & (low % 2 == 0), low, q)        # ... unless the lower is even
        q = q + 8 * np.signbit(g)
        q = np.where((amax == 0)[..., None] | bad[..., None], 0, q)
        scale = np.where(bad, 255, byte)
    return q.reshape(v.shape), scale


@pytest.mark.parametrize("fmt,group", [f for f in FORMATS if f[1]])
@pytest.mark.parametrize("rows,K", [(1, 128), (5, 384), (300, 1024)])
def test_quantizer(fmt, group, rows, K):
    rng = np.random.default_rng(rows + group)
    v = (rng.standard_normal((rows, K)) * 10.0 ** rng.integers(-39, 38, (rows, 1))
         ).astype(np.float32)
    v[0, :group] = 0
    if rows > 4:
        v[1, 3], v[2, group + 1], v[3, 0] = np.nan, np.inf, -np.inf
        v[4] = 0
        # ties of either grid: multiples of a quarter under a largest value of 6 or 7
        v[4, :group] = rng.integers(-24, 25, group) / 4
        v[4, 0] = 6 if fmt == "fp4" else 7
    t = bf16(v)
    got = ep.ep_quantize_w4(t.to(DEV), fmt, group)
    codes, scale = quantize_ref(t.float().numpy(), fmt, group)
    q = got.q.cpu().numpy()
    mine = np.stack([q & 15, q >> 4], -1).reshape(rows, K)
    zero = (mine == 8) & (codes == 0) if fmt == "fp4" else np.zeros_like(mine, bool)
    s = got.scale.float().cpu().numpy()
    assert np.array_equal(s, scale, equal_nan=True)
    assert ((mine == codes) | (zero & np.signbit(t.float().numpy()))).all()
    # half a step of the grid, by value
    ok = np.repeat(np.isfinite(scale) if fmt == "int4" else scale != 255, group, -1)
    back = w4_values(q, s.astype(np.float64) if fmt == "int4" else scale, fmt, group)
    top = np.repeat(np.abs(np.where(np.isfinite(v), t.float().numpy(), 0)).reshape(
        rows, -1, group).max(-1), group, -1)
    # int4: half of amax/7, a little more for the rounding of the scale; fp4: half of the
    # widest gap (2) of at most twice amax/6; and the least scales
    step = top * (0.5 / 7 * (1 + 2.0 ** -7) + 2.0 ** -8 if fmt == "int4" else 2.0 / 6) + 2.0 ** -127
    assert (np.abs(back - t.double().numpy())[ok] <= step[ok]).all()


@pytest.mark.parametrize("fmt", ["int4", "fp4"])
def test_quantizer_of_more_than_one_launch(fmt):
    """2^32 pieces of eight channels and a few more (69 GB of bf16): the rows at
    the ends and around the second launch's first piece as by themselves."""
    N, K = (1 << 20) + 3, 1 << 15
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    w = torch.zeros(N, K, dtype=torch.bfloat16, device=DEV)
    rows = [0, 1, N // 2, N - 6, N - 5, N - 4, N - 3, N - 2, N - 1]
    g = torch.Generator(device=DEV).manual_seed(2)
    w[rows] = torch.randn(len(rows), K, device=DEV, generator=g).to(torch.bfloat16)
    got = ep.ep_quantize_w4(w, fmt)
    alone = ep.ep_quantize_w4(w[rows], fmt)
    assert torch.equal(got.q[rows], alone.q) and torch.equal(got.scale[rows], alone.scale)
    nothing = 0x88 if fmt == "int4" else 0
    for r in (2, N // 4, N - 7):
        assert (got.q[r] == nothing).all()
        assert (got.scale[r] == 0).all()
    del w, got, alone
    torch.cuda.empty_cache()


def test_quantized_matrices_in_a_layer():
    """bf16 experts quantized by the package give the layer of their values."""
    rng = np.random.default_rng(21)
    T, K, E, H, I = 6, 2, 4, 256, 128
    w13, w2 = bf16(rng.standard_normal((E, 2 * I, H)) / 16), bf16(rng.standard_normal((E, H, I)) / 11)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, E)
    for fmt, group in FORMATS[1:]:
        a, b = (ep.ep_quantize_w4(t.to(DEV), fmt, group) for t in (w13, w2))
        vals = []
        for t in (a, b):
            s = t.scale.cpu().numpy() if fmt == "fp4" else f64(t.scale.cpu())
            v = w4_values(t.q.cpu().numpy(), s, fmt, group)
            vals += [v, np.abs(v) if fmt == "fp4" else 55 * np.repeat(s, group, -1)]
        out = ep.ep_moe_tokens(x.to(DEV), torch.from_numpy(idx).to(DEV),
                               torch.from_numpy(w).to(DEV), a, b)
        ref, tol = moe_ref(f64(x), idx, w, *vals, 0)
        check(out, ref, tol, fmt)
