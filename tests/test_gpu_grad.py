"""Gated activation with its 8-bit checkpoint, its backward pass and the
gradient of the combine, against plain 64-bit forms and differences."""

import numpy as np
import pytest
import torch

from oracle.epdc_oracle import bf16_to_f32, e4m3_encode
from tests.expert_helpers import BF16, STEP, TINY, bf16, check, f64
from tests.gpu_helpers import bits, gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

import combine_ep_send_amd as ep  # noqa: E402

DEV = "cuda:0"


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def quantize_ref(gu):
    """(codes, scales) by definition: scale = fl32(amax * fl32(1/448)) with NaN
    left out, code = e4m3(fl32(x / scale)); NaN gives 0x7F, and so does an
    infinity over its infinite scale."""
    v = bf16_to_f32(bits(gu)).reshape(gu.shape[0], -1, 128)
    amax = np.where(np.isnan(v), np.float32(0), np.abs(v)).max(-1)
    scale = (amax * np.float32(1 / 448)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        quo = v / scale[..., None]
        codes = np.where(np.isnan(quo), 0x7F, e4m3_encode(np.nan_to_num(quo)))
    zero = np.where(np.isnan(v), 0x7F, 0)
    codes = np.where((amax == 0)[..., None], zero, codes).astype(np.uint8)
    return codes.reshape(gu.shape), scale


def product_bound(g, value):
    """bf16 rounding, and (|g| + 8) 2^-22 relative for the sigmoid and the
    products; where exp(-g) leaves fp32 the sigmoid's 2^-126 is lost."""
    return BF16 * np.abs(value) + 1.01 * np.abs(value) * (np.abs(g) + 8) * 2.0 ** -22 + TINY


def act_ref(g, u):
    h = g * sigmoid(g) * u
    return h, product_bound(g, h) + np.abs(g * u) * 2.0 ** -125


def act_grad_ref(g, u, d):
    s = sigmoid(g)
    f = s * (1 + g * (1 - s))
    # the bracket may cancel: its error is relative to 1 + |g|
    ef = s * (1 + np.abs(g)) * (np.abs(g) + 8) * 2.0 ** -22 + (1 + np.abs(g)) * 2.0 ** -125
    dg, du = d * u * f, d * g * s
    tg = BF16 * np.abs(dg) + 1.01 * np.abs(d * u) * ef + 4 * STEP * np.abs(dg) + TINY
    tu = product_bound(g, du) + np.abs(d * g) * 2.0 ** -125
    return dg, tg, du, tu


def rows_of(rng, R, I):
    x = rng.standard_normal((R, 2 * I)) * rng.uniform(0.01, 8, (R, 1))
    if R > 2:
        x[1] *= 40                              # sigmoids of 0 and 1
        x[2, :128], x[2, I:I + 128] = 0, 0      # a group of zeros
        x[0] *= 1e-30
    return bf16(x)


@pytest.mark.parametrize("R,I", [(1, 128), (2, 384), (7, 256), (77, 512), (300, 128), (5, 2048)])
def test_activation_and_backward(R, I):
    rng = np.random.default_rng(R + I)
    gu, d = rows_of(rng, R, I), bf16(rng.standard_normal((R, I)))
    h, q, scale = ep.ep_swiglu_fp8(gu.to(DEV))
    v = f64(gu)
    ref, tol = act_ref(v[:, :I], v[:, I:])
    check(h, ref, tol, "h")
    oq, os = quantize_ref(gu)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), oq)
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), os.view(np.uint32))
    dgu, again = ep.ep_swiglu_fp8_backward(d.to(DEV), q, scale)
    kept = q.float().cpu().double().numpy() * np.repeat(os.astype(np.float64), 128, -1)
    g, u = kept[:, :I], kept[:, I:]
    dg, tg, du, tu = act_grad_ref(g, u, f64(d))
    check(dgu, np.concatenate([dg, du], 1), np.concatenate([tg, tu], 1), "gradient")
    ref, tol = act_ref(g, u)
    check(again, ref, tol, "h again")
    alone, none = ep.ep_swiglu_fp8_backward(d.to(DEV), q, scale, recompute=False)
    assert none is None and torch.equal(alone.view(torch.int16), dgu.view(torch.int16))


def test_activation_gradient_against_differences():
    """The formula used above is the derivative of silu(g) * u: central
    differences in 64 bits, error step^2 / 6 of the third derivative (< 1)."""
    rng = np.random.default_rng(3)
    g, u, d = rng.standard_normal((3, 4, 128)) * 3
    e = 1e-5
    dg, _, du, _ = act_grad_ref(g, u, d)
    num_g = d * (act_ref(g + e, u)[0] - act_ref(g - e, u)[0]) / (2 * e)
    num_u = d * (act_ref(g, u + e)[0] - act_ref(g, u - e)[0]) / (2 * e)
    assert np.abs(num_g - dg).max() < 1e-7 and np.abs(num_u - du).max() < 1e-7
    # and the kernel's gradient is the slope of the kernel's own definition at
    # the checkpoint's values, which codes that are exact make the input's
    R, I = 4, 128
    codes = rng.choice([-4, -2, -1.5, -1, -.5, .5, 1, 2, 3, 7], (R, 2 * I))
    codes[:, 0], codes[:, I] = 7, 7             # amax 7: scale 7/448 = 2^-6 (its product rounds to it)
    gu = bf16(codes)
    _, q, scale = ep.ep_swiglu_fp8(gu.to(DEV))
    got, h = ep.ep_swiglu_fp8_backward(bf16(d[:, :]).to(DEV), q, scale)
    v, dd = f64(gu), f64(bf16(d))
    num = np.concatenate([
        dd * (act_ref(v[:, :I] + e, v[:, I:])[0] - act_ref(v[:, :I] - e, v[:, I:])[0]) / (2 * e),
        dd * act_ref(v[:, :I], np.ones((R, I)))[0]], 1)
    dg, tg, du, tu = act_grad_ref(v[:, :I], v[:, I:], dd)
    check(got, num, np.concatenate([tg, tu], 1) + 1e-7)


@pytest.mark.parametrize("n", [0, 1, 5, 8, 9, -3])
def test_rows_past_the_count_are_left_alone(n):
    rng = np.random.default_rng(9)
    R, I = 8, 128
    gu, d = rows_of(rng, R, I).to(DEV), bf16(rng.standard_normal((R, I))).to(DEV)
    count = torch.tensor([n], dtype=torch.int32, device=DEV)
    use = min(max(n, 0), R)
    full = ep.ep_swiglu_fp8(gu)
    bufs = [torch.full_like(t.view(torch.uint8), 0x5A) for t in full]
    got = ep.ep_swiglu_fp8(gu, row_count=count, out=bufs[0].view(torch.bfloat16),
                           q=bufs[1].view(torch.float8_e4m3fn), scale=bufs[2].view(torch.float32))
    for b, f in zip(bufs, full):
        assert torch.equal(b[:use], f.view(torch.uint8)[:use]) and (b[use:] == 0x5A).all()
    back = ep.ep_swiglu_fp8_backward(d, full[1], full[2])
    bufs = [torch.full_like(t.view(torch.uint8), 0x5A) for t in back]
    ep.ep_swiglu_fp8_backward(d, full[1], full[2], row_count=count,
                              out=bufs[0].view(torch.bfloat16), h=bufs[1].view(torch.bfloat16))
    for b, f in zip(bufs, back):
        assert torch.equal(b[:use], f.view(torch.uint8)[:use]) and (b[use:] == 0x5A).all()
    assert got[0].data_ptr() != full[0].data_ptr()


def test_activation_of_values_that_are_not_finite():
    """NaN codes and infinite scales where the definition has them; other rows and other groups
    of the row are untouched."""
    rng = np.random.default_rng(10)
    R, I = 4, 256
    gu = rows_of(rng, R, I)
    gu[1, 5], gu[1, I + 130], gu[2, 200] = float("nan"), float("inf"), -float("inf")
    gu[3, 0:128] = float("nan")
    h, q, scale = ep.ep_swiglu_fp8(gu.to(DEV))
    with np.errstate(invalid="ignore"):
        oq, os = quantize_ref(gu)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), oq)
    assert np.array_equal(scale.cpu().numpy(), os, equal_nan=True)
    v = f64(gu)
    ok = np.isfinite(v[:, :I]) & np.isfinite(v[:, I:])
    ref, tol = act_ref(np.where(ok, v[:, :I], 0), np.where(ok, v[:, I:], 0))
    got = np.where(ok, h.double().cpu().numpy(), 0)
    check(got, ref, tol)
    assert not np.isfinite(h.double().cpu().numpy()[~ok]).any()


# ---------------------------------------------------------------------------
# combine
# ---------------------------------------------------------------------------

def rows_for(rng, T, K, P, unrouted):
    """token_row as a send layout makes it (slots of one destination share a
    row), and the row count."""
    dest = rng.integers(0, P, (T, K))
    dest[rng.random((T, K)) < unrouted] = -1
    row, n = np.full((T, K), -1, np.int32), 0
    for p in range(P):
        for t in range(T):
            at = dest[t] == p
            if at.any():
                row[t, at] = n
                n += 1
    return row, n


def combine_grad_ref(dout, y, row, w):
    R, H = y.shape
    T, K = row.shape
    dy, td = np.zeros((R, H)), np.zeros((R, H))
    dw, tw = np.zeros((T, K)), np.zeros((T, K))
    terms = 8 * (-(-H // 8192)) + 6 + 16 + 2    # longest chain: thread, lanes, waves
    for t in range(T):
        for k in range(K):
            r = row[t, k]
            if 0 <= r < R:
                dy[r] += (1.0 if w is None else float(w[t, k])) * dout[t]
                td[r] += (0.0 if w is None else abs(float(w[t, k]))) * np.abs(dout[t])
                dw[t, k] = dout[t] @ y[r]
                tw[t, k] = terms * STEP * (np.abs(dout[t]) @ np.abs(y[r])) + 2.0 ** -149
    return dy, BF16 * np.abs(dy) + (K + 1) * STEP * td + TINY, dw, tw


@pytest.mark.parametrize("T,K,P,H,unrouted", [
    (1, 1, 1, 8, 0.0), (5, 2, 2, 512, 0.0), (33, 3, 4, 72, 0.3), (16, 6, 8, 1000, 0.1),
    (9, 8, 3, 520, 0.2), (4, 16, 8, 264, 0.1), (3, 2, 2, 8192, 0.0), (3, 5, 4, 8200, 0.0),
    (2, 4, 2, 20000, 0.0), (40, 4, 40, 64, 1.0)])
def test_combine_backward(T, K, P, H, unrouted):
    rng = np.random.default_rng(T + K + H)
    row, R = rows_for(rng, T, K, P, unrouted)
    dout, y = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((R + 3, H)))
    w = rng.standard_normal((T, K)).astype(np.float32)
    d_row, d_w = torch.from_numpy(row).to(DEV), torch.from_numpy(w).to(DEV)
    dy, dw = ep.ep_combine_backward(dout.to(DEV), y.to(DEV), d_row, d_w)
    rdy, tdy, rdw, tdw = combine_grad_ref(f64(dout), f64(y), row, w)
    check(dy, rdy, tdy, "dy")
    check(dw, rdw, tdw, "dw")
    only, none = ep.ep_combine_backward(dout.to(DEV), None, d_row, d_w, weight_grad=False,
                                        num_rows=R + 3)
    assert none is None and torch.equal(only.view(torch.int16), dy.view(torch.int16))
    # unweighted: each row gets its token's gradient once, bit for bit
    buf = torch.full((R + 3, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_combine_backward(dout.to(DEV), None, d_row, None, dy=buf)
    want = torch.full((R + 3, H), 7.0, dtype=torch.bfloat16)
    for t in range(T):
        for r in row[t][row[t] >= 0]:
            want[r] = dout[t]
    assert torch.equal(buf.cpu(), want)


def test_combine_backward_against_differences():
    """The combine is linear in y and in w, so one difference in 64 bits of
    the plain combine gives the gradients the reference above states."""
    rng = np.random.default_rng(4)
    row, R = rows_for(rng, 6, 3, 2, 0.2)
    y, dout, w = rng.standard_normal((R, 4)), rng.standard_normal((6, 4)), rng.standard_normal((6, 3))

    def loss(y, w):
        return sum(w[t, k] * (y[row[t, k]] @ dout[t]) for t in range(6) for k in range(3)
                   if row[t, k] >= 0)
    dy, _, dw, _ = combine_grad_ref(dout, y, row, w)
    for r in range(R):
        for c in range(4):
            z = y.copy()
            z[r, c] += 1
            assert abs(loss(z, w) - loss(y, w) - dy[r, c]) < 1e-12
    for t in range(6):
        for k in range(3):
            v = w.copy()
            v[t, k] += 1
            assert abs(loss(y, v) - loss(y, w) - dw[t, k]) < 1e-12


def test_combine_backward_of_more_than_one_launch():
    """2^26 + 5 tokens of one wave each pass the work-items of one launch."""
    T, H = (1 << 26) + 5, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    dout = torch.randint(-4, 5, (T, H), device=DEV, generator=g, dtype=torch.int8
                         ).to(torch.bfloat16)
    y = torch.randint(-4, 5, (T, H), device=DEV, generator=g, dtype=torch.int8).to(torch.bfloat16)
    row = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)[:, None].contiguous()
    w = torch.randint(1, 4, (T, 1), device=DEV, generator=g).float()
    dy, dw = ep.ep_combine_backward(dout, y, row, w)
    # small integers: every product and sum is exact
    assert torch.equal(dy, (dout.float() * w).to(torch.bfloat16).flip(0))
    assert torch.equal(dw[:, 0], (dout.float() * y.flip(0).float()).sum(1))


def test_combine_backward_skips_rows_outside_the_buffer():
    rng = np.random.default_rng(5)
    T, K, H, R = 4, 3, 64, 5
    row = np.array([[0, 5, -1], [2 ** 31 - 1, -2 ** 31, 1], [4, 4, 4], [6, 7, 8]], np.int32)
    dout, y = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((R, H)))
    dout[3] = float("nan")                      # a token without a row
    w = rng.standard_normal((T, K)).astype(np.float32)
    w[0, 2] = np.nan                            # the weight of a slot without one
    buf = torch.full((R + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)
    dy, dw = ep.ep_combine_backward(dout.to(DEV), y.to(DEV), torch.from_numpy(row).to(DEV),
                                    torch.from_numpy(w).to(DEV), dy=buf[:R])
    rdy, tdy, rdw, tdw = combine_grad_ref(np.nan_to_num(f64(dout)), f64(y), row, np.nan_to_num(w))
    named = [0, 1, 4]
    check(dy[named], rdy[named], tdy[named])
    check(dw, rdw, tdw)
    assert (buf[[2, 3, 5]] == 7).all()


def test_activation_where_the_sigmoid_is_subnormal():
    """Gates of -87.5 to -88.5: 1 + exp(-g) lies past 2^126 and its reciprocal
    below the normal numbers, but not the product with a large u or dh."""
    R, I = 3, 128
    gate = np.array([-87.5, -88.0, -88.5])[:, None] * np.ones((R, I))
    rng = np.random.default_rng(11)
    u = np.ldexp(rng.uniform(1, 2, (R, I)), 118)
    gu = bf16(np.concatenate([gate, u], 1))
    d = bf16(rng.uniform(1, 2, (R, I)))

    def bound(g, value, factor):
        # as product_bound, but for the step of a subnormal sigmoid: 2^-149 and a half,
        # twice for the reciprocal's last place
        return BF16 * np.abs(value) + 1.01 * np.abs(value) * (np.abs(g) + 8) * 2.0 ** -22 + \
            np.abs(factor) * 2.0 ** -148
    h, q, scale = ep.ep_swiglu_fp8(gu.to(DEV))
    v = f64(gu)
    g, u = v[:, :I], v[:, I:]
    ref = g * sigmoid(g) * u
    assert np.abs(ref).min() > 2.0 ** -5
    check(h, ref, bound(g, ref, g * u), "h")
    dgu, again = ep.ep_swiglu_fp8_backward(d.to(DEV), q, scale)
    kept = q.float().cpu().double().numpy() * \
        np.repeat(scale.cpu().double().numpy(), 128, -1)
    # the values fp32 makes of code * scale
    kept = kept.astype(np.float32).astype(np.float64)
    g, u, d = kept[:, :I], kept[:, I:], f64(d)
    s = sigmoid(g)
    check(again, g * s * u, bound(g, g * s * u, g * u), "h again")
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    check(dgu[:, :I], dg, bound(g, dg, d * u * g), "dg")
    check(dgu[:, I:], du, bound(g, du, d * g) + TINY, "du")


def test_checkpoint_scale_is_pytorchs_quotient_on_the_gpu():
    """amax / 448.0 of a GPU tensor, which PyTorch computes as a product with
    the reciprocal: the same bits, over every exponent of bf16."""
    v = torch.arange(1, 0x7F80, dtype=torch.int16)                 # every positive finite value
    v = torch.cat([v, v[:128 * 256 - len(v)]]).view(torch.bfloat16).to(DEV)
    gu = torch.zeros(128, 2 * 16384, dtype=torch.bfloat16, device=DEV)
    gu[:, ::128] = v.view(128, 256)
    gu[:, 5::128] = -v.view(128, 256) / 2
    _, _, scale = ep.ep_swiglu_fp8(gu)
    amax = gu.float().view(128, 256, 128).abs().amax(-1)
    assert torch.equal(scale.view(torch.int32), (amax / 448.0).view(torch.int32))
