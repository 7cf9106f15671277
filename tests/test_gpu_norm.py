"""RMS norm with the residual's addition and the 8-bit output, and its gradient,
against 64 bits."""

import numpy as np
import pytest
import torch

import combine_ep_send_amd as ep
from tests.router_forms import (BF16, E4M3, F32, TINY, bf16, check, f64, norm_backward_ref,
                                norm_ref)

pytestmark = pytest.mark.gpu

# one token; odd rows; one lane's piece; a wave; several pieces a thread; past the
# workgroups of the backward; the most channels
SHAPES = [(1, 8), (1, 7168), (3, 128), (77, 520), (5, 4104), (1500, 256), (2, 16384), (2, 32768)]


def make(T, H, seed, f32, residual=True):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((T, H)) * rng.uniform(0.1, 4, (T, 1)))
    r = bf16(rng.standard_normal((T, H))) if residual else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(H))
    return rng, x, r, w.float() if f32 else w.to(torch.bfloat16)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_forward(T, H, f32):
    _, x, r, w = make(T, H, T + H, f32)
    n = ep.ep_rms_norm(x.cuda(), w.cuda(), 1e-5, residual=r.cuda(), rstd=True)
    s = (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(n.residual.cpu(), s)
    rstd, rtol, y, tol = norm_ref(f64(s), f64(w), float(np.float32(1e-5)))
    check(n.rstd, rstd, rtol, "rstd")
    check(n.y, y, tol + BF16 * np.abs(y) + TINY, "y")
    assert n.q is None and n.scale is None
    plain = ep.ep_rms_norm(s.cuda(), w.cuda(), 1e-5)
    assert torch.equal(plain.y, n.y) and plain.residual is None and plain.rstd is None


@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (77, 640), (3, 16384)])
@pytest.mark.parametrize("fmt", ["f32", "pow2"])
@pytest.mark.parametrize("f32", [False, True])
def test_codes_and_scales(T, H, fmt, f32):
    _, x, _, w = make(T, H, T * 3 + H, f32)
    both = ep.ep_rms_norm(x.cuda(), w.cuda(), fp8=True, scale_fmt=fmt)
    alone = ep.ep_rms_norm(x.cuda(), w.cuda(), fp8=True, bf16=False, scale_fmt=fmt)
    assert alone.y is None
    assert torch.equal(alone.q.view(torch.uint8), both.q.view(torch.uint8))
    assert torch.equal(alone.scale, both.scale)
    _, _, y, tol = norm_ref(f64(x), f64(w), float(np.float32(1e-6)))
    check(both.y, y, tol + BF16 * np.abs(y) + TINY, "y")
    amax = np.abs(y).reshape(T, -1, 128).max(-1) / 448
    near = (tol / np.maximum(np.abs(y), 1e-30)).max() + 2 * F32
    scale = f64(both.scale)
    if fmt == "f32":
        check(scale, amax, amax * near, "scale")
    else:
        assert (np.frexp(scale)[0] == 0.5).all()
        assert (scale >= amax * (1 - near)).all() and (scale < 2 * amax * (1 + near)).all()
    v = f64(both.q.float()).reshape(T, -1, 128) * scale[..., None]
    step = E4M3 * np.abs(y).reshape(v.shape) + 2.0 ** -10 * scale[..., None]
    check(v, y.reshape(v.shape), step * (1 + 1e-5) + tol.reshape(v.shape), "codes")


@pytest.mark.parametrize("fmt", ["f32", "pow2"])
@pytest.mark.parametrize("f32", [False, True])
def test_codes_are_the_roundings_of_64_bits(fmt, f32):
    """Whole numbers, whose squares' sums are exact: y is off by rounding in 64 bits alone,
    2^-50 of it, so scale and codes are the formula's roundings, unless a value lies
    within 2^-49 of a border.  About one value in 10^4 lies on the border of two codes
    but for the scale's rounding, so a scale one fp32 step off would show in codes."""
    rng = np.random.default_rng(17)
    T, H = 200, 1024
    x = rng.integers(-15, 16, (T, H)).astype(np.float64)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(H))
    w = w.float() if f32 else w.to(torch.bfloat16)
    n = ep.ep_rms_norm(bf16(x).cuda(), w.cuda(), 1e-6, fp8=True, scale_fmt=fmt)
    y = x / np.sqrt((x * x).mean(1, keepdims=True) + float(np.float32(1e-6))) * f64(w)
    y = y.reshape(T, -1, 128)
    ends = (1 - 2.0 ** -49, 1 + 2.0 ** -49)
    lo, hi = ((np.abs(y).max(-1) / 448 * e).astype(np.float32).astype(np.float64) for e in ends)
    if fmt == "pow2":
        lo, hi = (2.0 ** np.ceil(np.log2(v)) for v in (lo, hi))
    scale = f64(n.scale)
    assert ((lo <= scale) & (scale <= hi)).all() and (lo == hi).mean() > 0.99

    def code(v):
        v = np.clip(v, -448, 448).astype(np.float32)
        return torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    lo, hi = (code(y / scale[..., None] * e) for e in ends)
    got = f64(n.q.float()).reshape(y.shape)
    assert ((np.minimum(lo, hi) <= got) & (got <= np.maximum(lo, hi))).all()
    assert (lo == hi).mean() > 0.999


def test_codes_are_those_of_the_dispatch():
    """Rows that need no rounding on the way: signs times a power of two, rstd and
    weight powers of two, so that bf16 holds y and both quantizers see the same."""
    g = torch.Generator().manual_seed(1)
    T, H = 9, 512
    x = torch.where(torch.rand(T, H, generator=g) < 0.5, -1.0, 1.0)
    w = torch.exp2(torch.randint(-9, 4, (H,), generator=g).float()) * 1.375
    n = ep.ep_rms_norm(x.to(torch.bfloat16).cuda(), w.cuda(), 0.0, fp8=True)
    row = torch.arange(T, dtype=torch.int32)[:, None].cuda()
    q, scale = ep.ep_dispatch_permute(n.y, row, T, fp8=True)
    assert torch.equal(q.view(torch.uint8), n.q.view(torch.uint8))
    assert torch.equal(scale, n.scale)


def test_rows_of_zeros_infinities_and_nan():
    H = 256
    x = torch.ones(5, H)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 130] = float("nan")
    x[3, 128:] = 0.0
    x[4] = 1e-38
    w = torch.ones(H)
    w[200] = 0.0
    n = ep.ep_rms_norm(x.to(torch.bfloat16).cuda(), w.cuda(), 1e-6, fp8=True, rstd=True)
    y, q, scale = n.y.float().cpu(), n.q.view(torch.uint8).cpu(), n.scale.cpu()
    assert (y[0] == 0).all() and (q[0] == 0).all() and (scale[0] == 0).all()
    # an infinite mean square: rstd 0, so NaN at the infinity and 0 elsewhere
    assert n.rstd[1] == 0 and y[1, 3].isnan() and (y[1, :3] == 0).all()
    assert q[1, 3] == 0x7F and (q[1, 128:] == 0).all() and (scale[1] == 0).all()
    assert y[2].isnan().all() and (q[2] == 0x7F).all() and (scale[2] == 0).all()
    assert scale[3, 0] > 0 and scale[3, 1] == 0 and (q[3, 128:] == 0).all()
    # tiny rows beside eps: finite, scale at the bottom of fp32
    assert torch.isfinite(y[4]).all() and ((q[4] & 0x7F) != 0x7F).all()
    tiny = ep.ep_rms_norm(x[:1].to(torch.bfloat16).cuda() + 1, torch.full((H,), 1e-43).cuda(), 0.0,
                          fp8=True)
    # y is about 71 of fp32's least steps, amax / 448 rounds to none: zeros
    assert (tiny.scale == 0).all() and (tiny.q.view(torch.uint8) == 0).all()
    # 700 steps: a scale of 2 steps, quotients past 448 are cut to it
    tiny = ep.ep_rms_norm(x[:1].to(torch.bfloat16).cuda() + 1,
                          torch.full((H,), 700 * 2.0 ** -149).cuda(), 0.0, fp8=True)
    assert (tiny.scale == 2 * 2.0 ** -149).all()
    assert (tiny.q.float() == 352).all()            # 350 between 320 and 352


# mean squares that fp32 cannot hold, or holds in few bits; a bf16 number's square is
# exact in 64 bits
SIZES = [2.0 ** -132, 2.0 ** -110, 2.0 ** -80, 2.0 ** -75, 2.0 ** -70, 2.0 ** -66, 2.0 ** -50,
         2.0 ** 58, 2.0 ** 62, 2.0 ** 64, 2.0 ** 100, 2.0 ** 120]


@pytest.mark.parametrize("H", [8, 256, 640, 7168, 12288, 32768])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_of_every_size_without_eps(H, f32):
    """eps = 0 divides rows of every size by their own: y near the weight, whatever
    the size, with codes and without."""
    rng, x, _, w = make(len(SIZES), H, H, f32, False)
    x = bf16(f64(x) / np.sqrt((f64(x) ** 2).mean(1, keepdims=True)) *
             np.array(SIZES)[:, None])               # bf16's own least steps at the first
    least = torch.zeros(1, H, dtype=torch.bfloat16)
    least[0, H // 2] = TINY                          # the largest rstd there is
    x = torch.cat((x, least))
    fp8 = H % 128 == 0
    n = ep.ep_rms_norm(x.cuda(), w.cuda(), 0.0, fp8=fp8, rstd=True)
    rstd, rtol, y, tol = norm_ref(f64(x), f64(w), 0.0)
    held = rstd < torch.finfo(torch.float32).max     # the least rows' is past fp32
    assert held.sum() >= len(SIZES) - 1 and not held[-1]
    # the largest rows' is subnormal in fp32
    check(f64(n.rstd)[held], rstd[held], rtol[held] + 2.0 ** -150, "rstd")
    assert np.isinf(f64(n.rstd)[~held]).all()
    for got in (n.y, ep.ep_rms_norm(x.cuda(), w.cuda(), 0.0).y):
        check(got, y, tol + BF16 * np.abs(y) + TINY, "y")
    if fp8:
        scale = f64(n.scale)
        near = (tol / np.maximum(np.abs(y), 1e-30)).max() + 2 * F32
        amax = np.abs(y).reshape(len(x), -1, 128).max(-1) / 448
        check(scale, amax, amax * near, "scale")


@pytest.mark.parametrize("H", [256, 7168])
def test_backward_of_rows_of_every_size(H):
    """The first size's rstd is past fp32."""
    sizes = np.array(SIZES[1:])
    rng, s, _, w = make(len(sizes), H, H + 9, True, False)
    s = bf16(f64(s) / np.sqrt((f64(s) ** 2).mean(1, keepdims=True)) * sizes[:, None])
    dy = bf16(rng.standard_normal(s.shape))
    n = ep.ep_rms_norm(s.cuda(), w.cuda(), 0.0, rstd=True)
    dx, dw = ep.ep_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), n.rstd)
    rx, tx, rw, tw = norm_backward_ref(f64(dy), f64(s), f64(w), f64(n.rstd))
    check(dx, rx, tx, "dx")
    check(dw, rw, tw, "dw")


def test_rows_of_every_size_in_turn():
    """More rows than workgroups: a workgroup of two waves takes an ordinary row and
    then one of another size, or the other way round."""
    T, H = (1 << 20) + 4096, 520
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(T, H, device="cuda", generator=g)
    x *= torch.tensor([1.0, 2.0 ** -80, 2.0 ** 70, 2.0 ** -68, 3.0], device="cuda")[
        torch.arange(T, device="cuda") % 5, None]    # 2^20 leaves 1 over 5: sizes differ
    x = x.to(torch.bfloat16)
    w = torch.ones(H, device="cuda")
    n = ep.ep_rms_norm(x, w, 0.0)
    for r in torch.arange(T, device="cuda").split(1 << 17):
        s = x[r].double()
        y = s * s.square().mean(1, keepdim=True).rsqrt()
        # 64-bit values, or fp32 sums of eight squares, then two roundings
        assert bool(((n.y[r].double() - y).abs() <= (BF16 + 16 * F32) * y.abs()).all())


def test_rows_with_codes_and_without():
    """y from 64-bit values beside codes, from fp32 ones (four roundings) without: one
    bf16 step apart where a value lies that close to the border of two."""
    _, x, _, w = make(512, 2048, 14, True, False)
    a, b = (f64(ep.ep_rms_norm(x.cuda(), w.cuda(), fp8=fp8).y) for fp8 in (True, False))
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(a), np.abs(b)) + TINY)) - 7)
    assert (np.abs(a - b) <= step).all()
    # a border every 2^-8, at most 4 F32 of a value's size to either side of it
    assert (a != b).mean() < 2 * 8 * F32 / BF16
    both = a != b
    _, _, y, _ = norm_ref(f64(x), f64(w), float(np.float32(1e-6)))
    assert (np.abs(a - y)[both] <= (BF16 + F32) * np.abs(y)[both]).all()


def test_in_place_and_given_outputs():
    _, x, r, w = make(33, 1024, 5, False)
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    want = ep.ep_rms_norm(x, w, residual=r, fp8=True, rstd=True)
    r2 = r.clone()
    y = torch.empty_like(x)
    got = ep.ep_rms_norm(x, w, residual=r2, fp8=True, rstd=True, residual_out=r2, out=y,
                         q=torch.empty_like(want.q), scale=torch.empty_like(want.scale),
                         rstd_out=torch.empty_like(want.rstd))
    assert got.residual is r2 and got.y is y
    x2 = x.clone()
    over = ep.ep_rms_norm(x2, w, residual=r, residual_out=x2)
    for a, b in ((got.residual, want.residual), (got.y, want.y), (got.scale, want.scale),
                 (got.rstd, want.rstd), (got.q.view(torch.uint8), want.q.view(torch.uint8)),
                 (over.residual, want.residual),
                 (over.y, ep.ep_rms_norm(x, w, residual=r).y)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", SHAPES + [(4099, 512)])
@pytest.mark.parametrize("f32,residual", [(False, True), (True, False)])
def test_backward(T, H, f32, residual):
    rng, s, _, w = make(T, H, T + 2 * H, f32, False)
    dy, dr = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H)))
    rstd = 1 / np.sqrt((f64(s) ** 2).mean(1) + 1e-6)
    rstd32 = torch.from_numpy(rstd).float()
    dx, tol, dw, dtol = norm_backward_ref(f64(dy), f64(s), f64(w), f64(rstd32),
                                          f64(dr) if residual else None)
    got, gw = ep.ep_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), rstd32.cuda(),
                                      d_residual=dr.cuda() if residual else None)
    check(got, dx, tol, "dx")
    check(gw, dw, dtol, "dw")
    alone, none = ep.ep_rms_norm_backward(dy.cuda(), s.cuda(), w.cuda(), rstd32.cuda(),
                                          d_residual=dr.cuda() if residual else None,
                                          weight_grad=False)
    assert none is None and torch.equal(alone, got)


@pytest.mark.parametrize("H,f32", [(4096, False), (8192, True), (12288, False), (24576, True)])
def test_rows_past_the_cache(H, f32):
    """Inputs of 384 MiB and more, which are read past the caches, with a residual: every
    row as a call of few rows gives it, rows at both ends against 64 bits."""
    T = (384 << 20) // (4 * H) + 5
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    x, r, dy = (torch.randn(T, H, device="cuda", generator=g).bfloat16() for _ in range(3))
    w = 1 + 0.3 * torch.randn(H, device="cuda", generator=g)
    w = w if f32 else w.bfloat16()
    few = [slice(a, min(a + 2000, T)) for a in range(0, T, 2000)]
    for fp8 in (False, True):
        n = ep.ep_rms_norm(x, w, 1e-5, residual=r, fp8=fp8, rstd=True)
        for b in few:
            m = ep.ep_rms_norm(x[b], w, 1e-5, residual=r[b], fp8=fp8, rstd=True)
            assert torch.equal(n.residual[b], m.residual) and torch.equal(n.rstd[b], m.rstd)
            assert torch.equal(n.y[b], m.y)
            if fp8:
                assert torch.equal(n.q[b].view(torch.uint8), m.q.view(torch.uint8))
                assert torch.equal(n.scale[b], m.scale)
        for b in (slice(0, 2), slice(T - 2, T)):
            s = (x[b].float() + r[b].float()).bfloat16()
            assert torch.equal(n.residual[b], s)
            _, _, y, tol = norm_ref(f64(s), f64(w), float(np.float32(1e-5)))
            check(n.y[b], y, tol + BF16 * np.abs(y) + TINY, "y")
    dx, dw = ep.ep_rms_norm_backward(dy, n.residual, w, n.rstd, d_residual=r)
    want, size = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in few:
        m, _ = ep.ep_rms_norm_backward(dy[b], n.residual[b], w, n.rstd[b], d_residual=r[b])
        assert torch.equal(dx[b], m)
        part = dy[b].double() * n.residual[b].double() * n.rstd[b].double()[:, None]
        want, size = want + part.sum(0), size + part.abs().sum(0)
    # as in norm_backward_ref
    assert bool(((dw - want).abs() <= (T / 256 + 86) * F32 * size).all())


def test_backward_in_place_and_no_tokens():
    rng, s, _, w = make(50, 264, 8, False, False)
    dy, dr = bf16(rng.standard_normal((50, 264))).cuda(), bf16(rng.standard_normal((50, 264))).cuda()
    s, w = s.cuda(), w.cuda()
    rstd = ep.ep_rms_norm(s, w, rstd=True).rstd
    want, dw = ep.ep_rms_norm_backward(dy, s, w, rstd, d_residual=dr)
    over = dr.clone()
    got, dw2 = ep.ep_rms_norm_backward(dy, s, w, rstd, d_residual=over, out=over)
    assert got is over and torch.equal(got, want) and torch.equal(dw, dw2)
    over = dy.clone()
    got, _ = ep.ep_rms_norm_backward(over, s, w, rstd, d_residual=dr, out=over)
    assert torch.equal(got, want)
    none, dw = ep.ep_rms_norm_backward(dy[:0], s[:0], w, rstd[:0], dw=torch.ones(264).cuda())
    assert none.shape == (0, 264) and (dw == 0).all()
    empty = ep.ep_rms_norm(s[:0], w, residual=s[:0])
    assert empty.y.shape == empty.residual.shape == (0, 264)


def test_gradient_against_differences():
    """The gradient of sum(c * y) along a direction, from the forward itself in
    64-bit sums.  The forward's bf16 output is off by 2^-8 of a value at each end;
    what is left is of second order in the step."""
    rng, x, r, w = make(4, 512, 21, True)
    c, v = bf16(rng.standard_normal((4, 512))), rng.standard_normal((4, 512))
    n = ep.ep_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), rstd=True)
    dx, _ = ep.ep_rms_norm_backward(c.cuda(), n.residual, w.cuda(), n.rstd)
    s, h = f64(n.residual), 1e-4

    def value(a):
        rstd = 1 / np.sqrt((a * a).mean(1) + 1e-6)
        return (f64(c) * a * rstd[:, None] * f64(w)).sum()
    slope = (value(s + h * v) - value(s - h * v)) / (2 * h)
    got = (f64(dx) * v).sum()
    # dx's rounding, element by element, and the differences' own
    assert abs(got - slope) <= 1.1 * BF16 * np.abs(f64(dx) * v).sum() + 1e-5


@pytest.mark.parametrize("H", [512, 4104])
def test_gradient_of_a_cotangent_along_the_row(H):
    """Cotangents close to the normalised row, so that dx is what the mean leaves of a ten
    times larger g: along the row nothing (y does not change with the row's size, but
    for eps), along others what central differences of the formula in 64 bits give, their
    error of third order in the step.  Row by row, within dx's rounding, which dx without
    the mean's term, or with its other sign, is far outside of."""
    rng, s, _, w = make(6, H, H + 2, True, False)
    w64, eps = f64(w), float(np.float32(1e-6))
    n = ep.ep_rms_norm(s.cuda(), w.cuda(), 1e-6, rstd=True)
    s64, rstd = f64(s), f64(n.rstd)[:, None]
    c = bf16(s64 * rstd / w64 + 0.1 * rng.standard_normal((6, H)))
    dx, _ = ep.ep_rms_norm_backward(c.cuda(), s.cuda(), w.cuda(), n.rstd)
    dx, c = f64(dx), f64(c)
    term = rstd * s64 * rstd * (c * w64 * s64 * rstd).mean(1, keepdims=True)

    def value(a):
        return (c * w64 * a / np.sqrt((a * a).mean(1, keepdims=True) + eps)).sum(1)
    for v in (s64, rng.standard_normal((6, H)) / rstd):
        h = 1e-5
        slope = (value(s64 + h * v) - value(s64 - h * v)) / (2 * h)
        # dx's rounding to bf16; fp32 roundings of the two terms it is the difference of,
        # 92 additions for the mean's; the differences' own: 64-bit values over the step
        tol = BF16 * np.abs(dx * v).sum(1) + 100 * F32 * np.abs(term * v).sum(1) + \
            2.0 ** -50 * np.abs(c * w64 * s64 * rstd).sum(1) / h + 1e-8 * np.abs(c * v).sum(1)
        assert (np.abs((dx * v).sum(1) - slope) <= tol).all()
        for wrong in (dx + term, dx + 2 * term):
            assert (np.abs((wrong * v).sum(1) - slope) > 5 * tol).any()
    assert (np.abs(((dx + term) * s64).sum(1)) > 50 * BF16 * np.abs(dx * s64).sum(1)).all()


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16).cuda()
    w = torch.ones(256).cuda()
    for kw, match in ((dict(bf16=False), "asked"), (dict(residual_out=x), "residual"),
                      (dict(q=x), "fp8"), (dict(rstd_out=w), "rstd"), (dict(scale_fmt="ue8m0", fp8=True), "scale_fmt"),
                      (dict(residual=x[:3]), "shape"), (dict(residual=x.float()), "bfloat16"),
                      (dict(out=x.t()), "contiguous"), (dict(bf16=False, fp8=True, out=x), "bf16"),
                      (dict(eps=-1.0), "argument"), (dict(eps=float("inf")), "argument")):
        with pytest.raises(ValueError, match=match):
            ep.ep_rms_norm(x, w, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_rms_norm(x[:, ::2], w[:128])
    with pytest.raises(ValueError, match="shape"):
        ep.ep_rms_norm(x, w[:128])
    with pytest.raises(ValueError, match="128"):
        ep.ep_rms_norm(x[:, :8].contiguous(), w[:8], fp8=True)
    with pytest.raises(ValueError):
        ep.ep_rms_norm(x[:, :12].contiguous(), w[:12])
    with pytest.raises(ValueError, match="workspace"):
        ep.ep_rms_norm_backward(x, x, w, w[:4], workspace=torch.empty(8, dtype=torch.uint8).cuda())
    with pytest.raises(ValueError, match="weight_grad"):
        ep.ep_rms_norm_backward(x, x, w, w[:4], weight_grad=False, dw=w)
