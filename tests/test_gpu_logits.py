"""The router's logits and their gradients against 64 bits."""

import numpy as np
import pytest
import torch

import combine_ep_send_amd as ep
from tests.router_forms import DEEP, bf16, check, f64, logits_backward_ref, logits_ref

pytestmark = pytest.mark.gpu

# one token and one expert; tiles that end inside; each number of rows and
# experts a workgroup takes; channels split over workgroups or not; several
# workgroups of experts
SHAPES = [(1, 1, 8), (1, 256, 7168), (3, 8, 512), (16, 64, 256), (17, 60, 1000), (33, 130, 2056),
          (65, 7, 4096), (130, 256, 264), (257, 64, 520), (20, 1024, 1032), (9, 300, 65536),
          (4200, 128, 320), (4200, 250, 136), (4160, 64, 72), (9000, 96, 64)]


def make(T, E, H, seed):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((T, H)))
    w = bf16(rng.standard_normal((E, H)) / np.sqrt(H))
    return rng, x, w


@pytest.mark.parametrize("T,E,H", SHAPES)
def test_logits(T, E, H):
    _, x, w = make(T, E, H, T + E + H)
    got = ep.ep_router_logits(x.cuda(), w.cuda())
    check(got, *logits_ref(f64(x), f64(w)))


@pytest.mark.parametrize("T,E,H", SHAPES)
def test_backward(T, E, H):
    rng, x, w = make(T, E, H, 2 * T + E + H)
    dl = (rng.standard_normal((T, E)) * rng.uniform(0.01, 10, (T, 1))).astype(np.float32)
    d = torch.from_numpy(dl).cuda()
    dx, dw = ep.ep_router_logits_backward(d, x.cuda(), w.cuda())
    rx, tx, rw, tw = logits_backward_ref(dl.astype(np.float64), f64(x), f64(w))
    check(dx, rx, tx, "dx")
    check(dw, rw, tw, "dw")
    only, none = ep.ep_router_logits_backward(d, None, w.cuda(), weight_grad=False)
    assert none is None and torch.equal(only, dx)
    none, only = ep.ep_router_logits_backward(d, x.cuda(), None, input_grad=False)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("T,E,H", DEEP)
def test_many_stages_are_exact(T, E, H):
    """Whole numbers whose sums of magnitudes fit fp32's 24 bits: equal to the bit in
    whatever order, so that a stage taken twice, left out or read too early shows."""
    rng = np.random.default_rng(T + E + H)
    x, w = (rng.integers(-8, 9, (n, H)).astype(np.float64) for n in (T, E))
    assert 64 * H < 1 << 24
    got = ep.ep_router_logits(bf16(x).cuda(), bf16(w).cuda())
    assert np.array_equal(f64(got), x @ w.T)
    # 12 bits: two bf16 parts
    d = rng.integers(-(1 << 11), (1 << 11) + 1, (T, E)).astype(np.float64)
    x[rng.random((T, H)) < 0.9] = 0.0
    x, w = np.sign(x), np.clip(w, -2, 2)
    assert (np.abs(d).T @ np.abs(x)).max() < 1 << 24 and 4096 * E < 1 << 24
    dx, dw = ep.ep_router_logits_backward(torch.from_numpy(d).float().cuda(), bf16(x).cuda(),
                                          bf16(w).cuda())
    assert torch.equal(dx.cpu(), bf16(d @ w))
    assert np.array_equal(f64(dw), d.T @ x)


@pytest.mark.parametrize("T,E,H", DEEP)
def test_many_stages(T, E, H):
    rng, x, w = make(T, E, H, T + 2 * E + H)
    check(ep.ep_router_logits(x.cuda(), w.cuda()), *logits_ref(f64(x), f64(w)))
    dl = (rng.standard_normal((T, E)) * rng.uniform(0.01, 10, (T, 1))).astype(np.float32)
    dx, dw = ep.ep_router_logits_backward(torch.from_numpy(dl).cuda(), x.cuda(), w.cuda())
    rx, tx, rw, tw = logits_backward_ref(dl.astype(np.float64), f64(x), f64(w))
    check(dx, rx, tx, "dx")
    check(dw, rw, tw, "dw")


def test_small_numbers_are_exact():
    """Whole numbers whose sums fit fp32: every product and sum is exact, whatever
    the order, and the parts of the logits' gradient are too (17 bits and up)."""
    rng = np.random.default_rng(2)
    T, E, H = 100, 72, 648
    x, w = rng.integers(-8, 9, (T, H)), rng.integers(-8, 9, (E, H))
    got = ep.ep_router_logits(bf16(x * 1.0).cuda(), bf16(w * 1.0).cuda())
    assert np.array_equal(f64(got), x @ w.T)
    dl = rng.integers(-(1 << 20), 1 << 20, (T, E))
    one = np.sign(rng.integers(-3, 4, (T, H)))
    one[rng.random((T, H)) < 0.9] = 0                # few terms: sums below 2^24
    _, dw = ep.ep_router_logits_backward(torch.from_numpy(dl).float().cuda(),
                                         bf16(one * 1.0).cuda(), None, input_grad=False)
    keep = np.abs(dl).T @ np.abs(one) < 1 << 24
    assert keep.mean() > 0.5
    assert np.array_equal(f64(dw)[keep], (dl.T @ one)[keep])


def test_infinities_and_nan_stay_in_their_rows():
    _, x, w = make(40, 20, 256, 6)
    x[3, 7], x[5, 0] = float("nan"), float("inf")
    w[11, 9] = float("nan")
    got = ep.ep_router_logits(x.cuda(), w.cuda()).cpu()
    assert got[3].isnan().all() and got[:, 11].isnan().all()
    assert not got[5, :11].isfinite().any()
    rest = np.delete(np.delete(f64(got), [3, 5], 0), 11, 1)
    ref, tol = logits_ref(np.delete(f64(x), [3, 5], 0), np.delete(f64(w), 11, 0))
    check(rest, ref, tol)
    d = torch.randn(40, 20)
    d[2, 4], d[9, 6] = float("inf"), float("nan")
    d[12, 1] = 3.4e38                                # past the largest bf16: finite all the same
    _, x, w = make(40, 20, 256, 7)
    dx, dw = ep.ep_router_logits_backward(d.cuda(), x.cuda(), w.cuda())
    bad = [2, 9]
    rx, tx, rw, tw = logits_backward_ref(f64(d), f64(x), f64(w))
    check(np.delete(f64(dx), bad, 0), np.delete(rx, bad, 0), np.delete(tx, bad, 0))
    check(np.delete(f64(dw), [4, 6, 1], 0), np.delete(rw, [4, 6, 1], 0),
          np.delete(tw, [4, 6, 1], 0))
    assert not dx.cpu()[bad].isfinite().any() and dw.cpu()[6].isnan().all()
    # an infinity takes part as one, not as a NaN
    assert torch.equal(dw.cpu()[4], torch.where(x[2].float() > 0, float("inf"), -float("inf")))


@pytest.mark.parametrize("T,E,H", [(40, 20, 264), (300, 130, 72)])
def test_largest_gradients(T, E, H):
    """Finite gradients that bf16 would round to infinities, times small numbers:
    finite results, as near as others are."""
    _, x, w = make(T, E, H, 10)
    x, w = x * 2.0 ** -8, w * 2.0 ** -8              # exact; sums stay below 2^127
    d = torch.zeros(T, E)
    d[3, 1], d[8, 5] = torch.finfo(torch.float32).max, -3.39616e38 - 1e34
    d[9, 5] = 3.3962e38
    d[11, 7] = torch.finfo(torch.bfloat16).max
    dx, dw = ep.ep_router_logits_backward(d.cuda(), x.cuda(), w.cuda())
    rx, tx, rw, tw = logits_backward_ref(f64(d), f64(x), f64(w))
    check(dx, rx, tx, "dx")
    check(dw, rw, tw, "dw")


@pytest.mark.parametrize("T,E,H", [(40, 20, 264), (300, 130, 72)])
def test_backward_of_infinite_rows_and_weights(T, E, H):
    """What meets an infinity is none or NaN, as the header says; nothing else is."""
    rng, x, w = make(T, E, H, 11)
    d = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    dx, dw = ep.ep_router_logits_backward(d.cuda(), x.cuda(), w.cuda())
    x[4, 9], w[6, 13] = float("inf"), -float("inf")
    bx, bw = ep.ep_router_logits_backward(d.cuda(), x.cuda(), w.cuda())
    assert not bx[:, 13].isfinite().any() and not bw[:, 9].isfinite().any()
    rest = [h for h in range(H) if h != 13]
    assert torch.equal(bx[:, rest], dx[:, rest])
    rest = [h for h in range(H) if h != 9]
    assert torch.equal(bw[:, rest], dw[:, rest])


@pytest.mark.parametrize("T,E,H", [(2100, 200, 328), (2100, 200, 584), (40, 20, 264)])
def test_infinite_weights(T, E, H):
    """An infinite weight in the last channels, whose stage ends before its products
    do: infinities of x's sign in its expert's column, the others as they were."""
    _, x, w = make(T, E, H, 8)
    x[x == 0] = 1.0
    want = ep.ep_router_logits(x.cuda(), w.cuda()).cpu()
    w[7, H - 1], w[9, 2] = float("inf"), -float("inf")
    got = ep.ep_router_logits(x.cuda(), w.cuda()).cpu()
    inf = torch.tensor(float("inf"))
    assert torch.equal(got[:, 7], torch.where(x[:, H - 1].float() > 0, inf, -inf))
    assert torch.equal(got[:, 9], torch.where(x[:, 2].float() > 0, -inf, inf))
    keep = [e for e in range(E) if e not in (7, 9)]
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("T,E,H", [(70, 64, 264), (2100, 200, 328)])
def test_arrays_aligned_to_four_bytes(T, E, H):
    rng, x, w = make(T, E, H, 9)
    x, w = x.cuda(), w.cuda()
    room = torch.full((T * E + 2,), 7.0).cuda()
    out = room[1:-1].view(T, E)
    assert torch.equal(ep.ep_router_logits(x, w, out=out), ep.ep_router_logits(x, w))
    assert room[0] == 7 and room[-1] == 7
    d = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    out.copy_(d)
    for a, b in zip(ep.ep_router_logits_backward(out, x, w), ep.ep_router_logits_backward(d, x, w)):
        assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    """More than 2^31 channels in all: the last rows as computed alone."""
    T, E, H = 300001, 160, 7168
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    w = (torch.randn(E, H, device="cuda") / 85).bfloat16()
    tail = slice(T - 70, T)
    y = ep.ep_router_logits(x, w)
    check(y[tail], *logits_ref(f64(x[tail]), f64(w)))
    d = torch.randn(T, E, device="cuda")
    dx, dw = ep.ep_router_logits_backward(d, x, w)
    alone, _ = ep.ep_router_logits_backward(d[tail].contiguous(), None, w, weight_grad=False)
    assert torch.equal(dx[tail], alone)
    # the sums over all rows, against fp32 sums of 64-bit ones over runs of them
    want = torch.zeros(E, H, dtype=torch.float64, device="cuda")
    size = torch.zeros(E, H, dtype=torch.float64, device="cuda")
    for r in torch.arange(T, device="cuda").split(20000):
        want += d[r].double().t() @ x[r].double()
        size += d[r].double().abs().t() @ x[r].double().abs()
    tol = (2.0 ** -24 + (3 * T / 32 + 96) * 2.0 ** -23) * size
    assert bool(((dw.double() - want).abs() <= tol).all())
    del x, d, dx, y
    n = 330000
    s = torch.empty(n, 7168, dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.ones(7168, device="cuda")
    a, b = ep.ep_rms_norm(s, g, fp8=True, rstd=True), ep.ep_rms_norm(s[-9:].contiguous(), g, fp8=True)
    assert torch.equal(a.y[-9:], b.y) and torch.equal(a.scale[-9:], b.scale)
    assert torch.equal(a.q[-9:].view(torch.uint8), b.q.view(torch.uint8))
    back, _ = ep.ep_rms_norm_backward(s, s, g, a.rstd)
    last, _ = ep.ep_rms_norm_backward(s[-9:].contiguous(), s[-9:].contiguous(), g,
                                      a.rstd[-9:].contiguous())
    assert torch.equal(back[-9:], last)


def test_no_tokens_given_outputs_and_refusals():
    _, x, w = make(10, 12, 128, 1)
    x, w, d = x.cuda(), w.cuda(), torch.randn(10, 12).cuda()
    out = torch.empty(10, 12).cuda()
    assert ep.ep_router_logits(x, w, out=out) is out
    assert torch.equal(out, ep.ep_router_logits(x, w))
    assert ep.ep_router_logits(x[:0], w).shape == (0, 12)
    dx, dw = ep.ep_router_logits_backward(d[:0], x[:0], w, dw=torch.ones(12, 128).cuda())
    assert dx.shape == (0, 128) and (dw == 0).all()
    ws = torch.empty(ep.ep_router_logits_backward_workspace_bytes(10, 12, 128),
                     dtype=torch.uint8).cuda()
    a = ep.ep_router_logits_backward(d, x, w)
    b = ep.ep_router_logits_backward(d, x, w, workspace=ws, dx=torch.empty_like(x),
                                     dw=torch.empty(12, 128).cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for fn, match in ((lambda: ep.ep_router_logits(x, w[:, :64].contiguous()), "channels"),
                      (lambda: ep.ep_router_logits(x, w.float()), "bfloat16"),
                      (lambda: ep.ep_router_logits(x, w, workspace=ws[:16]), "workspace"),
                      (lambda: ep.ep_router_logits(x[:, ::2], w), "contiguous"),
                      (lambda: ep.ep_router_logits_backward(d, x, None), "needs w"),
                      (lambda: ep.ep_router_logits_backward(d, None, w), "needs x"),
                      (lambda: ep.ep_router_logits_backward(d, x, w, workspace=ws[256:]), "workspace"),
                      (lambda: ep.ep_router_logits_backward(d, x, w, input_grad=False,
                                                            weight_grad=False), "asked"),
                      (lambda: ep.ep_router_logits_backward(d, x, w, input_grad=False, dx=x), "input_grad")):
        with pytest.raises(ValueError, match=match):
            fn()
