"""The choice of a token's experts and the gradient of its weights, against 64
bits: the ids exactly, the weights to one rounding."""

import numpy as np
import pytest
import torch

import combine_ep_send_amd as ep
from tests.router_forms import F32, SMALL, check, f64, route_backward_ref, route_ref

pytestmark = pytest.mark.gpu


def run(l, K, bias=None, count=None, **kw):
    idx, w = ep.ep_route(torch.from_numpy(l).cuda(), K,
                         bias=None if bias is None else torch.from_numpy(bias).cuda(),
                         token_count=None if count is None else
                         torch.tensor([count], dtype=torch.int32).cuda(), **kw)
    return idx.cpu().numpy(), f64(w)


def against(l, K, bias=None, count=None, score="softmax", num_groups=1, topk_groups=1, group_top=2,
            renormalize=True, scale=1.0):
    idx, w = run(l, K, bias, count, score=score, num_groups=num_groups, topk_groups=topk_groups,
                 group_top=group_top, renormalize=renormalize, scale=scale)
    ri, rw = route_ref(l.astype(np.float64), K, score, None if bias is None else
                       bias.astype(np.float64), num_groups, topk_groups, group_top, renormalize,
                       scale, count)
    assert np.array_equal(idx, ri), np.argwhere(idx != ri)[:5]
    check(w, rw, np.abs(rw) * F32 * (1 + 1e-6) + SMALL, "weights")
    return idx, w


def logits(T, E, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    return rng, (spread * rng.standard_normal((T, E))).astype(np.float32)


# every width of the lanes' lists: experts to 16, 32, 64, 128, 256, 512, 1024
@pytest.mark.parametrize("E", [1, 2, 8, 17, 60, 64, 127, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("K", [1, 2, 3, 8, 11, 16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_and_slots(E, K, score):
    rng, l = logits(21, E, E * 17 + K)
    against(l, K, score=score)
    against(l, K, (0.1 * rng.standard_normal(E)).astype(np.float32), score=score, scale=2.5,
            renormalize=K % 2 == 0)


@pytest.mark.parametrize("E,G,kept", [(16, 16, 3), (60, 4, 2), (64, 8, 3), (96, 12, 5), (256, 8, 4),
                                      (255, 15, 4), (272, 16, 1), (160, 5, 3), (1024, 8, 4),
                                      (1017, 9, 4), (8, 2, 1), (512, 2, 1)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_groups(E, G, kept, top, score, biased):
    rng, l = logits(19, E, E + G + kept + top)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if biased else None
    against(l, min(8, E), bias, score=score, num_groups=G, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 1000])
def test_tokens(T):
    _, l = logits(T, 33, T)
    against(l, 4, renormalize=False)


def test_more_tokens_than_one_launch_takes():
    """16 tokens a workgroup of 256: 2^28 and some take two launches."""
    T = (1 << 28) + 77
    l = torch.zeros(T, 2, device="cuda")
    l[T - 100:, 1] = 1.0
    l[:9, 1] = 2.0
    idx, w = ep.ep_route(l, 1)
    assert bool((w == 1).all()) and int(idx.sum()) == 109
    assert bool((idx[T - 100:] == 1).all()) and bool((idx[:9] == 1).all())
    d = ep.ep_route_backward(w, l, idx, score="sigmoid", renormalize=False)
    at = torch.tensor([0, 9, (1 << 28) - 1, 1 << 28, T - 1], device="cuda")
    s = torch.sigmoid(l[at].double().gather(1, idx[at]))[:, 0]
    got = d[at].double()
    check(got.gather(1, idx[at])[:, 0], f64(s * (1 - s)), f64(s) * F32)
    assert bool((got.gather(1, 1 - idx[at]) == 0).all())


def test_ties_go_to_the_lowest_number():
    l = np.zeros((3, 40), np.float32)
    l[1] = np.repeat(np.arange(10, dtype=np.float32), 4)
    l[2, ::2] = -0.0                                 # equal to +0
    for kw in (dict(), dict(score="sigmoid"), dict(bias=np.zeros(40, np.float32)),
               dict(num_groups=8, topk_groups=3), dict(num_groups=8, topk_groups=3, group_top=1),
               dict(score="sigmoid", bias=np.full(40, -3, np.float32), num_groups=4, topk_groups=2)):
        idx, _ = against(l, 6, **kw)
        assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]


def test_neighbouring_logits_are_told_apart():
    """Logits one step of fp32 apart, about 1 and about 2^-120, in scores and
    without: 32-bit scores would tie and order by number."""
    for base in (1.0, 2.0 ** -120, -3.0):
        steps = np.arange(64, dtype=np.int32)
        l = (np.float32(base).view(np.int32) + steps).view(np.float32)[None].repeat(2, 0).copy()
        l[1] = l[1, ::-1]
        against(l, 16)
        if abs(base) >= 1:
            # scores apart by 2^-26 and more of their size
            against(l, 16, np.zeros(64, np.float32))
            against(l, 16, np.zeros(64, np.float32), score="sigmoid")


@pytest.mark.parametrize("base", [8.0, 13.0, -20.0, -80.0])
def test_neighbouring_large_logits_are_told_apart(base):
    """Sigmoids of logits one fp32 step apart: up to 13 they differ by 2^-39 and more, and
    keys are held to 2^-43 below 1; negative ones by 2^-20 of their size."""
    steps = np.arange(64, dtype=np.int32)
    l = (np.float32(base).view(np.int32) + steps).view(np.float32)[None].repeat(2, 0).copy()
    l[1] = l[1, ::-1]
    against(l, 16, np.zeros(64, np.float32), score="sigmoid")
    against(l, 16, score="sigmoid")
    against(l, 16, score="sigmoid", num_groups=4, topk_groups=2)


def test_saturated_sigmoids_are_equal_keys():
    """From 40 on a sigmoid is 1 in 64 bits: with a bias the lowest numbers win, without one
    the logits still order."""
    l = np.linspace(40, 90, 32, dtype=np.float32)[None].repeat(2, 0).copy()
    l[1] = l[1, ::-1]
    idx, w = against(l, 4, np.zeros(32, np.float32), score="sigmoid")
    assert (idx == [0, 1, 2, 3]).all() and (w == 0.25).all()
    idx, w = against(l, 4, score="sigmoid")
    assert idx.tolist() == [[31, 30, 29, 28], [0, 1, 2, 3]] and (w == 0.25).all()


def test_masked_experts_and_empty_rows():
    rng, l = logits(12, 48, 3)
    low = np.finfo(np.float32).min
    l[0] = -np.inf                                   # nothing left
    l[1, 3:] = -np.inf                               # fewer experts than slots
    l[2] = np.nan
    l[3, ::2] = np.nan
    l[4] = low                                       # the lowest value is no mask: all equal
    l[5, 1:] = low
    l[6, :40] = -np.inf                              # whole groups away
    l[7, 5] = np.inf
    l[8] = -200.0                                    # sigmoids of 2^-288: below fp32
    l[9] = -800.0                                    # below 64 bits too
    bias = (0.1 * rng.standard_normal(48)).astype(np.float32)
    bias[7], bias[9], bias[11] = -np.inf, np.nan, np.inf
    for kw in (dict(), dict(renormalize=False), dict(score="sigmoid"),
               dict(score="sigmoid", renormalize=False), dict(bias=bias, score="sigmoid"),
               dict(bias=bias), dict(num_groups=6, topk_groups=2, score="sigmoid"),
               dict(num_groups=6, topk_groups=2, group_top=1)):
        idx, w = run(l, 6, **kw)
        ref = dict(kw)
        ri, rw = route_ref(l.astype(np.float64), 6, ref.pop("score", "softmax"),
                           ref.pop("bias", None), ref.get("num_groups", 1),
                           ref.get("topk_groups", 1), ref.get("group_top", 2),
                           ref.get("renormalize", True))
        assert np.array_equal(idx, ri), (kw, np.argwhere(idx != ri)[:5])
        assert np.array_equal(np.isnan(w), np.isnan(rw)), kw
        fin = ~np.isnan(rw)
        check(np.where(fin, w, 0), np.where(fin, rw, 0),
              np.where(fin, np.abs(rw) * F32 * 1.001, 0) + SMALL, str(kw))
        assert (idx[0] == -1).all() and (w[0] == 0).all() and (idx[2] == -1).all()


def test_padding_tokens_are_not_routed():
    _, l = logits(40, 24, 9)
    l[30:] = np.nan
    for count in (0, 1, 16, 30, 40, 100, -5):
        idx, w = run(l[:30] if count > 30 else l, 3, count=count)
        ri, rw = route_ref((l[:30] if count > 30 else l).astype(np.float64), 3, count=count)
        assert np.array_equal(idx, ri)
        check(w, rw, np.abs(rw) * F32 * 1.001 + SMALL)


@pytest.mark.parametrize("E,G", [(24, 1), (64, 4), (600, 1), (1024, 8)])
def test_workgroups_of_padding(E, G):
    """Counts inside a workgroup's tokens (16, or 4 past 256 experts), at their ends and
    with whole workgroups behind them; what the outputs held is overwritten."""
    rng, l = logits(70, E, E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    d, b = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    kw = dict(score="sigmoid", bias=b, num_groups=G, topk_groups=max(1, G // 2))
    want_idx, want_w = ep.ep_route(d, 5, **kw)
    for count in (-3, 0, 1, 3, 4, 5, 15, 16, 17, 31, 32, 64, 69, 70, 71):
        n = min(70, max(0, count))
        pad = d.clone()
        pad[n:] = float("nan")
        idx = torch.full((70, 5), 77, device="cuda")
        w = torch.full((70, 5), 7.0, device="cuda")
        ep.ep_route(pad, 5, token_count=torch.tensor([count], dtype=torch.int32).cuda(),
                    topk_idx=idx, topk_weights=w, **kw)
        assert torch.equal(idx[:n], want_idx[:n]) and torch.equal(w[:n], want_w[:n]), count
        assert bool((idx[n:] == -1).all()) and bool((w[n:] == 0).all()), count


@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (60, 4), (127, 16), (256, 8), (300, 8), (1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward(E, K, score, renorm):
    rng, l = logits(37, E, E + K)
    K = min(K, E)
    idx = np.argsort(rng.random((37, E)), axis=1)[:, :K].astype(np.int64)
    idx[rng.random((37, K)) < 0.2] = -1
    idx[3] = -1
    idx[4, 0], idx[5, 0] = E, -7                     # no experts either
    dw = rng.standard_normal((37, K)).astype(np.float32)
    got = ep.ep_route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(l).cuda(),
                               torch.from_numpy(idx).cuda(), score=score, renormalize=renorm,
                               scale=1.5)
    ref, tol = route_backward_ref(dw.astype(np.float64), l.astype(np.float64), idx, score, renorm,
                                  1.5)
    check(got, ref, tol)
    assert (got[3] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_repeated_and_masked_experts(score, renorm):
    rng, l = logits(6, 20, 77)
    idx = np.array([[3, 3, 5, 3], [7, 7, 7, 7], [0, 1, 2, 2], [-1, 4, -1, 4], [0, 5, 6, 7],
                    [-1, -1, -1, -1]], np.int64)
    l[4, :] = -np.inf
    l[4, :6] = 0.5                                   # experts 6 and 7 are masked: no weight
    l[5] = np.nan                                    # a token without slots: zeros all the same
    dw = rng.standard_normal((6, 4)).astype(np.float32)
    got = ep.ep_route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(l).cuda(),
                               torch.from_numpy(idx).cuda(), score=score, renormalize=renorm)
    ref, tol = route_backward_ref(dw.astype(np.float64), l.astype(np.float64), idx, score, renorm)
    check(got, ref, tol)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(score, renorm):
    """The weights' change along a direction, by central differences of the
    formula in 64 bits; their error is of third order in the step."""
    rng, l = logits(5, 32, 4)
    idx, _ = run(l, 4, score=score, renormalize=renorm)
    dw, v = rng.standard_normal((5, 4)).astype(np.float32), rng.standard_normal((5, 32))

    def value(a):
        from tests.router_forms import scores64
        s = np.take_along_axis(scores64(a, score), idx, 1)
        return (dw * s / (s.sum(1, keepdims=True) if renorm else 1)).sum()
    h = 1e-5
    slope = (value(l + h * v) - value(l - h * v)) / (2 * h)
    got = ep.ep_route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(l).cuda(),
                               torch.from_numpy(idx).cuda(), score=score, renormalize=renorm)
    assert abs((f64(got) * v).sum() - slope) <= F32 * np.abs(f64(got) * v).sum() + 1e-8


@pytest.mark.parametrize("top", [-700.0, -709.5, -712.0, -720.0, -735.0])
def test_backward_of_sigmoids_near_the_least_number(top):
    """Renormalised weights of scores that 64 bits only just hold: the reciprocal of
    their sum, which 64 bits do not, takes no part.  The shares are the formula's,
    from logits less the largest; a score's rounding to a multiple of 2^-1074 is a part
    2^-1075 / s of it, and a share has two of them."""
    rng = np.random.default_rng(int(-top))
    T, E, K = 9, 24, 5
    l = (top - 4.0 * rng.random((T, E))).astype(np.float32)
    l[8] = -800.0                                    # a sum of 0: no gradient
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int64)
    idx[0, 1:] = -1                                  # one slot: a constant weight
    idx[1, 3] = idx[1, 2]
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = ep.ep_route_backward(torch.from_numpy(dw).cuda(), torch.from_numpy(l).cuda(),
                               torch.from_numpy(idx).cuda(), score="sigmoid", scale=2.0)
    ref, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(8):
        ks = idx[t] >= 0
        e, d = idx[t, ks], 2.0 * dw[t, ks].astype(np.float64)
        q = np.exp(l[t, e].astype(np.float64) - l[t, e].max())
        q /= q.sum()                                 # 1 - s is 1 here
        np.add.at(ref[t], e, q * (d - (d * q).sum()))
        np.add.at(size[t], e, q * (np.abs(d) + np.abs(d * q).sum()))
    least = 2.0 ** -1074 / np.exp(top - 4.0)
    check(got, ref, F32 * np.abs(ref) + (2.0 ** -44 + 4 * least) * size + SMALL)


@pytest.mark.parametrize("scale", [2.0 ** -30, 1e-3, 1.0, 2.5])
@pytest.mark.parametrize("top", [-700.0, -712.0, -735.0])
def test_weights_of_sigmoids_near_the_least_number(top, scale):
    """Renormalised weights of scores that 64 bits only just hold, scaled up and down:
    the scale takes no bits from them.  A score's rounding as in the test above."""
    rng = np.random.default_rng(int(-top))
    l = (top - 4.0 * rng.random((9, 24))).astype(np.float32)
    idx, w = run(l, 5, score="sigmoid", scale=scale)
    assert np.array_equal(idx, np.argsort(-l, axis=1, kind="stable")[:, :5])
    at = np.take_along_axis(l, idx, 1).astype(np.float64)
    q = np.exp(at - at[:, :1])
    q *= float(np.float32(scale)) / q.sum(1, keepdims=True)
    check(w, q, (F32 + 2.0 ** -44 + 2 * 2.0 ** -1074 / np.exp(top - 4.0)) * q, "weights")


def test_arrays_aligned_to_four_bytes():
    """Logits and bias off by a float: the loads of fours need 16 bytes."""
    rng, l = logits(50, 64, 2)
    room, bias = torch.zeros(50 * 64 + 1).cuda(), torch.zeros(65).cuda()
    off = room[1:].view(50, 64)
    off.copy_(torch.from_numpy(l))
    bias[1:] = torch.from_numpy((0.1 * rng.standard_normal(64)).astype(np.float32)).cuda()
    even = off.clone(), bias[1:].clone()
    for kw in (dict(), dict(num_groups=4, topk_groups=2)):
        for a, b in ((off, bias[1:]), (off, even[1]), (even[0], bias[1:])):
            got = ep.ep_route(a, 6, score="sigmoid", bias=b, **kw)
            want = ep.ep_route(even[0], 6, score="sigmoid", bias=even[1], **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_given_outputs_and_refusals():
    _, l = logits(9, 16, 1)
    d = torch.from_numpy(l).cuda()
    want = ep.ep_route(d, 2)
    idx, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = ep.ep_route(d, 2, topk_idx=idx, topk_weights=w)
    assert got[0] is idx and torch.equal(idx, want[0]) and torch.equal(w, want[1])
    assert ep.ep_route(d[:0], 2)[0].shape == (0, 2)
    assert ep.ep_route_backward(w[:0], d[:0], idx[:0]).shape == (0, 16)
    # more slots than experts: the rest is unrouted
    idx, w = ep.ep_route(d[:, :3].contiguous(), 8)
    assert (idx[:, 3:] == -1).all() and (w[:, 3:] == 0).all() and (idx[:, :3] >= 0).all()
    for kw in (dict(num_topk=0), dict(num_topk=17), dict(num_topk=2, score="tanh"),
               dict(num_topk=2, num_groups=3), dict(num_topk=2, num_groups=4, topk_groups=5),
               dict(num_topk=2, num_groups=4, topk_groups=2, group_top=3),
               dict(num_topk=2, scale=float("nan")), dict(num_topk=1 << 40),
               dict(num_topk=2, bias=d[0, :8]), dict(num_topk=2, bias=d[0].double()),
               dict(num_topk=2, token_count=idx[0, :1]), dict(num_topk=2, num_groups=1 << 33)):
        with pytest.raises(ValueError):
            ep.ep_route(d, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_route(d[:, ::2], 2)
    with pytest.raises(ValueError, match="float32"):
        ep.ep_route(d.bfloat16(), 2)
