"""The calls before the dispatch as they are used: rows in 8 bits through the
dispatch, a layer's front into dispatch and combine, its training step, graphs,
streams."""

import numpy as np
import pytest
import torch

import combine_ep_send_amd as ep
from tests.router_forms import (BF16, TINY, bf16, check, f64, logits_backward_ref,
                                norm_backward_ref, permute_ref, route_ref)

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def codes(g, T, H):
    return torch.randint(0, 256, (T, H), dtype=torch.uint8, generator=g)


# one word of scales a row; rows of several chunks; scales in 16-byte pieces and not
@pytest.mark.parametrize("T,H,K", [(1, 128, 1), (7, 512, 2), (40, 640, 3), (33, 1024, 4),
                                   (9, 7168, 6), (50, 2048, 8), (21, 4224, 16)])
@pytest.mark.parametrize("offset", [0, 1])
def test_quantized_rows_move_unchanged(T, H, K, offset):
    g = torch.Generator().manual_seed(T + H + K)
    cap, W = T * K + 3, H // 128
    q, scale = codes(g, T, H), torch.randint(-(1 << 31), 1 << 31, (T, W), generator=g).int()
    row = torch.randperm(cap, generator=g)[:T * K].view(T, K).int()
    row[torch.rand(T, K, generator=g) < 0.2] = -1
    if K > 1:
        row[:, 1] = row[:, 0]                        # two slots of one destination
    row[0, -1] = cap                                 # outside
    held_q, held_s = codes(g, cap, H), torch.rand(cap, W, generator=g)
    # an offset of one float: scales that are not 16-byte aligned
    room, out_room = torch.zeros(T * W + 1).cuda(), torch.zeros(cap * W + 1).cuda()
    s = room[offset:offset + T * W].view(T, W)
    s.copy_(scale.view(torch.float32))
    out_scale = out_room[offset:offset + cap * W].view(cap, W)
    out_scale.copy_(held_s)
    out = held_q.cuda().view(FP8)
    got, got_s = ep.ep_dispatch_permute_quantized(q.cuda().view(FP8), s, row.cuda(), cap, out=out,
                                                  out_scale=out_scale)
    assert got is out and got_s is out_scale
    assert np.array_equal(got.view(torch.uint8).cpu().numpy(),
                          permute_ref(q.numpy(), row.numpy(), held_q.numpy()))
    assert np.array_equal(got_s.view(torch.int32).cpu().numpy(),
                          permute_ref(scale.numpy(), row.numpy(), held_s.view(torch.int32).numpy()))


@pytest.mark.parametrize("words", [0, 1, 3, 8, 700])
def test_rows_with_any_number_of_scale_words(words):
    """The C call moves as many words a row as it is told: none, other groups' scales."""
    from combine_ep_send_amd import _lib

    g = torch.Generator().manual_seed(words)
    T, H, K, cap = 37, 256, 3, 130
    q = codes(g, T, H)
    scale = torch.randint(-(1 << 31), 1 << 31, (T, words), generator=g).int()
    row = torch.randperm(cap, generator=g)[:T * K].view(T, K).int()
    held_q, held_s = codes(g, cap, H), torch.full((cap, words), 5, dtype=torch.int32)
    dq, ds, dr, out, out_s = (t.cuda() for t in (q, scale, row, held_q, held_s))
    st = _lib.lib().ep_dispatch_permute_quantized(
        dq.data_ptr(), ds.data_ptr() if words else None, words, T, H, dr.data_ptr(), K, cap,
        out.data_ptr(), out_s.data_ptr() if words else None,
        torch.cuda.current_stream().cuda_stream)
    assert st == _lib.EP_OK
    assert np.array_equal(out.cpu().numpy(), permute_ref(q.numpy(), row.numpy(), held_q.numpy()))
    assert np.array_equal(out_s.cpu().numpy(),
                          permute_ref(scale.numpy(), row.numpy(), held_s.numpy()))


def test_quantized_rows_past_one_launch():
    """128 channels a row: 33.6 M tokens take two launches of 2^32 - 1 work-items."""
    T = (1 << 25) + 1001
    q = torch.empty(T, 32, dtype=torch.int32, device="cuda").random_()
    scale = torch.arange(T, dtype=torch.float32, device="cuda")[:, None].contiguous()
    row = (torch.arange(T, dtype=torch.int32, device="cuda") + 12345) % T
    out, out_scale = ep.ep_dispatch_permute_quantized(q.view(FP8), scale, row[:, None].contiguous(),
                                                      T)
    out = out.view(torch.int32)
    assert torch.equal(out[12345:], q[:-12345]) and torch.equal(out[:12345], q[-12345:])
    assert torch.equal(out_scale[12345:], scale[:-12345])
    assert torch.equal(out_scale[:12345], scale[-12345:])


def routed(T, E, K, seed):
    g = torch.Generator().manual_seed(seed)
    idx, w = ep.ep_route(torch.randn(T, E, generator=g).cuda(), K)
    idx[torch.rand(T, K, generator=g).cuda() < 0.1] = -1
    return idx, w


@pytest.mark.parametrize("num_send", [None, 400])
def test_dispatch_of_quantized_rows(num_send):
    """The same received rows as from bf16 rows quantized on the way."""
    idx, w = routed(100, 32, 4, 1)
    x = torch.randn(100, 1024).to(torch.bfloat16).cuda()
    same = torch.arange(100, dtype=torch.int32)[:, None].cuda()
    q, scale = ep.ep_dispatch_permute(x, same, 100, fp8=True)
    kw = dict(num_local_experts=4, num_ranks=8, num_send=num_send)
    (aq, as_), ai, aw, ah = ep.dispatch(x, idx, w, fp8=True, **kw)
    (bq, bs), bi, bw, bh = ep.dispatch((q, scale), idx, w, **kw)
    n = int(ah.send_counts.sum())
    assert torch.equal(aq.view(torch.uint8)[:n], bq.view(torch.uint8)[:n])
    assert torch.equal(as_[:n], bs[:n]) and torch.equal(ai[:n], bi[:n])
    assert torch.equal(ah.token_row, bh.token_row)


@pytest.mark.parametrize("streams,exact", [(1, False), (2, False), (2, True)])
def test_chunked_dispatch_of_quantized_rows(streams, exact):
    idx, w = routed(130, 32, 4, 2)
    x = torch.randn(130, 512).to(torch.bfloat16).cuda()
    same = torch.arange(130, dtype=torch.int32)[:, None].cuda()
    q, scale = ep.ep_dispatch_permute(x, same, 130, fp8=True)
    d = ep.ChunkedDispatcher(130, 4, 512, num_local_experts=4, num_ranks=8, chunks=3, fp8=True,
                             streams=streams, exact_counts=exact)

    def local(_, recv, *rest):
        codes_, sc = recv
        return (codes_.float().unflatten(-1, (-1, 128)) * sc[..., None]).flatten(-2).bfloat16()
    want = d.forward(x, idx, w, local).clone()
    got = d.forward((q, scale), idx, w, local)
    assert torch.equal(want, got)
    assert torch.equal(want, ep.dispatch_chunked_forward(
        (q, scale), idx, w, lambda *a: local(0, *a), num_local_experts=4, num_ranks=8, chunks=3,
        fp8=True))
    with pytest.raises(ValueError, match="scales"):
        d.forward((q, scale[:, :2]), idx, w, local)
    plain = ep.ChunkedDispatcher(130, 4, 512, num_local_experts=4, num_ranks=8, chunks=3)
    with pytest.raises(ValueError, match="fp8"):
        plain.forward((q, scale), idx, w, local)


class Front:
    """A layer from the residual stream to the combine, experts left out."""

    def __init__(self, T, H, E, K, P, seed, fp8):
        g = torch.Generator().manual_seed(seed)
        self.K, self.E, self.P, self.fp8 = K, E, P, fp8
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.residual = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.weight = (1 + 0.2 * torch.randn(H, generator=g)).cuda()
        self.gate = (torch.randn(E, H, generator=g) * H ** -0.5).to(torch.bfloat16).cuda()
        self.bias = (0.05 * torch.randn(E, generator=g)).cuda()

    def forward(self, count=None):
        n = ep.ep_rms_norm(self.x, self.weight, residual=self.residual, fp8=self.fp8, rstd=True)
        logits = ep.ep_router_logits(n.y, self.gate)
        idx, w = ep.ep_route(logits, self.K, score="sigmoid", bias=self.bias, num_groups=4,
                             topk_groups=2, scale=1.5, token_count=count)
        recv, ridx, rw, handle = ep.dispatch((n.q, n.scale) if self.fp8 else n.y, idx, w,
                                             num_local_experts=self.E // self.P, num_ranks=self.P,
                                             num_send=idx.shape[0] * min(self.K, self.P))
        if self.fp8:
            recv = (recv[0].float().unflatten(-1, (-1, 128)) * recv[1][..., None]).flatten(-2)
            recv = recv.to(torch.bfloat16)
        return n, logits, idx, w, recv, handle, ep.combine(recv, handle)

    def backward(self, dout, n, logits, idx, recv, handle):
        d_local, d_w = ep.combine_backward(dout, recv, handle)
        d_logits = ep.ep_route_backward(d_w, logits, idx, score="sigmoid", scale=1.5)
        d_y, d_gate = ep.ep_router_logits_backward(d_logits, n.y, self.gate)
        # the rows' gradient from both users of y, summed in fp32
        d_y = ep.ep_combine(d_local, handle.token_row, None, bias=d_y)
        dx, d_weight = ep.ep_rms_norm_backward(d_y, n.residual, self.weight, n.rstd, d_residual=dout)
        return d_w, d_logits, d_gate, d_y, dx, d_weight


def test_front_of_a_layer():
    f = Front(75, 512, 32, 4, 8, 11, True)
    n, logits, idx, w, _, handle, out = f.forward()
    y = f64(n.y)
    check(logits, y @ f64(f.gate).T, 56 * 2.0 ** -23 * (np.abs(y) @ np.abs(f64(f.gate)).T))
    ri, rw = route_ref(f64(logits), 4, "sigmoid", f64(f.bias), 4, 2, scale=1.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    check(w, rw, np.abs(rw) * 2.0 ** -23)
    # every slot's row is the token's in 8 bits: the combine scales it by the weights' sum
    row = f64(n.q.float()) * np.repeat(f64(n.scale), 128, 1)
    ref = row * f64(w).sum(1, keepdims=True)
    check(out, ref, 2.1 * BF16 * np.abs(ref) + TINY)


def test_padding_reaches_no_expert():
    f = Front(64, 256, 16, 2, 4, 3, False)
    f.x[40:] = float("nan")
    count = torch.tensor([40], dtype=torch.int32).cuda()
    n, logits, idx, w, _, handle, out = f.forward(count)
    assert (idx[40:] == -1).all() and (w[40:] == 0).all() and (out[40:] == 0).all()
    assert out[:40].isfinite().all() and (handle.token_row[40:] == -1).all()


def test_training_step_against_autograd():
    """Every gradient of a step, against autograd in 64 bits on the values that the
    forward kept, the choice being constant."""
    f = Front(90, 256, 32, 4, 8, 5, False)
    n, logits, idx, w, recv, handle, out = f.forward()
    dout = bf16(np.random.default_rng(1).standard_normal((90, 256))).cuda()
    d_w, d_logits, d_gate, d_y, dx, d_weight = f.backward(dout, n, logits, idx, recv, handle)
    y = n.y.double().cpu().requires_grad_()
    gate = f.gate.double().cpu().requires_grad_()
    l = y @ gate.t()
    s = torch.sigmoid(l).gather(1, idx.cpu())
    wt = 1.5 * s / s.sum(1, keepdim=True)
    l.retain_grad()
    wt.retain_grad()
    ((wt.sum(1, keepdim=True) * y) * dout.double().cpu()).sum().backward()
    # wt's sum is constant, so what reaches the router cancels: bounds count sizes.  The
    # slots' gradients are sums of 256 products in fp32, their mean goes off again.
    size = (np.abs(f64(dout)) * np.abs(f64(n.y))).sum(1, keepdims=True)
    check(d_w, f64(wt.grad), 300 * 2.0 ** -24 * size + 1e-30)
    e = 320 * 2.0 ** -24 * 1.5 * size
    check(d_logits, f64(l.grad), np.broadcast_to(e, l.shape))
    check(d_gate, f64(gate.grad), np.broadcast_to(1.1 * (e * np.abs(f64(n.y))).sum(0), gate.shape))
    # d_y: rows rounded to bf16 by the combine's gradient (one for each of up to four rows),
    # then once more in the sum
    rows = np.abs(f64(wt).sum(1, keepdims=True) * f64(dout))
    tol = BF16 * (2.1 * rows + np.abs(f64(y.grad))) + 40 * e * np.abs(f64(f.gate)).max() + TINY
    check(d_y, f64(y.grad), tol)
    # the norm's backward, from the d_y that reached it
    s = n.residual.double().cpu().requires_grad_()
    weight = f.weight.double().cpu().requires_grad_()
    z = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * weight
    (z * d_y.double().cpu()).sum().backward()
    rx = f64(s.grad) + f64(dout)
    g = np.abs(f64(d_y) * f64(f.weight)) * f64(n.rstd)[:, None]
    m = np.abs(f64(n.y)) * (g.mean(1, keepdims=True) + 1)
    check(dx, rx, BF16 * np.abs(rx) + 200 * 2.0 ** -24 * (g + m * (1 + g.mean(1, keepdims=True))) * 4)
    check(d_weight, f64(weight.grad),
          300 * 2.0 ** -24 * np.abs(f64(d_y) * f64(n.residual) * f64(n.rstd)[:, None]).sum(0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_every_gradient_of_a_step(score, renorm):
    """As the step above, with experts that differ: each destination scales its rows by a
    power of two of its own (exact in bf16), so that renormalised weights have a gradient
    too.  Every gradient is far larger than its bound, so that zeros, another scale or a
    share left out would not pass.  The last tokens are padding."""
    T, H, E, K, P, live = 90, 256, 32, 4, 8, 84
    f = Front(T, H, E, K, P, 6, False)
    factor = torch.tensor([1.0, -2.0, 0.5, 4.0, -1.0, 2.0, -0.5, 1.0]).cuda()
    how = dict(score=score, renormalize=renorm, scale=1.5)
    n = ep.ep_rms_norm(f.x, f.weight, residual=f.residual, rstd=True)
    logits = ep.ep_router_logits(n.y, f.gate)
    idx, w = ep.ep_route(logits, K, bias=f.bias, num_groups=4, topk_groups=2,
                         token_count=torch.tensor([live], dtype=torch.int32).cuda(), **how)
    recv, _, _, handle = ep.dispatch(n.y, idx, w, num_local_experts=E // P, num_ranks=P)
    by = factor[handle.send_rank.long()][:, None].bfloat16()
    local = recv * by
    out = ep.combine(local, handle)
    dout = bf16(np.random.default_rng(2).standard_normal((T, H))).cuda()
    d_local, d_w = ep.combine_backward(dout, local, handle)
    d_logits = ep.ep_route_backward(d_w, logits, idx, **how)
    d_router, d_gate = ep.ep_router_logits_backward(d_logits, n.y, f.gate)
    d_y = ep.ep_combine(d_local * by, handle.token_row, None, bias=d_router)

    y = n.y.double().cpu().requires_grad_()
    gate = f.gate.double().cpu().requires_grad_()
    some = torch.arange(T)[:, None] < live
    at = idx.cpu().clamp(min=0)
    assert torch.equal(idx.cpu() >= 0, some.expand(T, K))
    l = y @ gate.t()
    s = (torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)).gather(1, at)
    wt = 1.5 * s / s.sum(1, keepdim=True) if renorm else 1.5 * s
    for t in (l, wt):
        t.retain_grad()
    scale = factor.double().cpu()[at // (E // P)] * some
    res = (wt * scale).sum(1, keepdim=True) * y
    (res * dout.double().cpu()).sum().backward()

    def seen(ref, tol):
        # half of them at least: tokens whose experts share a factor have no gradient
        # where weights are renormalised
        part = float((np.abs(ref) > 10 * tol).mean())
        assert part > 0.5
    weights, ys, gs = f64(wt.detach()), np.abs(f64(n.y)), np.abs(f64(f.gate))
    fs = np.abs(scale.numpy())
    # a row's factor is exact; up to K rows are added in fp32 and rounded once
    check(out, f64(res.detach()), BF16 * np.abs(f64(res.detach())) +
          8 * 2.0 ** -24 * (weights * fs).sum(1, keepdims=True) * ys + TINY, "out")
    # sums of H products in fp32
    e = 300 * 2.0 ** -24 * (np.abs(f64(dout)) * ys).sum(1, keepdims=True)
    check(d_w, f64(wt.grad), e * fs + 1e-30, "d_w")
    seen(f64(wt.grad)[:live], (e * fs)[:live])
    # a weight's share of its logit's gradient is at most scale, twice: its own and the mean's
    worst = 3 * e * fs.max(1, keepdims=True)
    tol = worst + 2.0 ** -24 * np.abs(f64(l.grad))
    check(d_logits, f64(l.grad), tol, "d_logits")
    seen(f64(l.grad.gather(1, at))[:live], tol[:live].max(1, keepdims=True))
    # the router's products from the d_logits that reached them, and with that one's bound
    # against autograd
    rx, tx, rw, tw = logits_backward_ref(f64(d_logits), f64(n.y), f64(f.gate))
    check(d_gate, rw, tw, "d_gate")
    seen(rw, tw)
    check(d_gate, f64(gate.grad), tw + np.broadcast_to(tol, (T, E)).T @ ys, "d_gate by autograd")
    # the router's share, rounded to bf16 (in tx); a destination's rows, each rounded to
    # bf16; their sum in fp32, rounded
    ref, size = rx.copy(), np.abs(rx)
    for r in range(P):
        hit = (at.numpy() // (E // P) == r) & some.numpy()
        row = (weights * scale.numpy() * hit).sum(1, keepdims=True) * f64(dout)
        ref, size = ref + row, size + np.abs(row)
    near = tx + BF16 * 1.01 * size + BF16 * np.abs(ref) + TINY
    check(d_y, ref, near, "d_y")
    seen(ref[:live], near[:live])
    seen(rx[:live], 0.3 * near[:live])
    check(d_y, f64(y.grad), near + np.broadcast_to(tol, (T, E)) @ gs, "d_y by autograd")
    # the norm's, from the d_y that reached it
    dx, d_weight = ep.ep_rms_norm_backward(d_y, n.residual, f.weight, n.rstd, d_residual=dout)
    rx, tx, rw, tw = norm_backward_ref(f64(d_y), f64(n.residual), f64(f.weight), f64(n.rstd),
                                       f64(dout))
    check(dx, rx, tx, "dx")
    check(d_weight, rw, tw, "d_weight")
    seen(rw, tw)


def test_layer_of_a_few_tokens():
    """The serving form: norm, router and ep_moe_tokens, three tokens."""
    g = torch.Generator().manual_seed(4)
    H, I, E = 256, 128, 16
    x = torch.randn(3, H, generator=g).to(torch.bfloat16).cuda()
    weight = torch.ones(H).cuda()
    gate = (torch.randn(E, H, generator=g) / 16).to(torch.bfloat16).cuda()
    w13 = (torch.randn(E, 2 * I, H, generator=g) / 16).to(torch.bfloat16).cuda()
    w2 = (torch.randn(E, H, I, generator=g) / 16).to(torch.bfloat16).cuda()
    n = ep.ep_rms_norm(x, weight)
    idx, w = ep.ep_route(ep.ep_router_logits(n.y, gate), 2)
    out = ep.ep_moe_tokens(n.y, idx, w, w13, w2)
    y, ref, mag = f64(n.y), np.zeros((3, H)), np.zeros((3, H))
    ri, rw = route_ref(y @ f64(gate).T, 2)
    assert np.array_equal(idx.cpu().numpy(), ri)
    for t in range(3):
        for k in range(2):
            gu = f64(w13[ri[t, k]]) @ y[t]
            h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            ref[t] += rw[t, k] * (f64(w2[ri[t, k]]) @ h)
            mag[t] += rw[t, k] * (np.abs(f64(w2[ri[t, k]])) @ np.abs(h))
    check(out, ref, BF16 * np.abs(ref) + 2.0 ** -13 * mag)


@pytest.mark.parametrize("fp8", [False, True])
def test_replayed_graphs(fp8):
    """Two captured steps replayed in turn with other inputs, eager work between:
    each replay equals the eager result, so the graphs share nothing."""
    fronts = [Front(96, 512, 32, 4, 8, 20 + i, fp8) for i in range(2)]
    dout = torch.randn(96, 512).to(torch.bfloat16).cuda()

    def step(f):
        n, logits, idx, w, recv, handle, out = f.forward()
        return (n.y, n.residual, logits, idx, w, out, *f.backward(dout, n, logits, idx, recv, handle))
    for f in fronts:
        step(f)
    side = torch.cuda.Stream()
    graphs = []
    for f in fronts:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(f)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kept = step(f)
        graphs.append((f, g, kept))
    for i in range(4):
        for f, g, kept in graphs:
            f.x.copy_(torch.randn(96, 512, generator=torch.Generator().manual_seed(i)).bfloat16())
            g.replay()
        for f, g, kept in graphs:
            for a, b in zip(kept, step(f)):
                assert torch.equal(a, b)
        torch.cuda.synchronize()
    ep.check_workspaces()


def test_another_stream_and_two_at_once():
    a, b = Front(200, 1024, 64, 8, 8, 30, True), Front(333, 1024, 64, 8, 8, 31, True)
    want = [f.forward() for f in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for f, s in zip((a, b), streams):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for f, s in zip((a, b), streams):
            n = ep.ep_rms_norm(f.x, f.weight, residual=f.residual, fp8=True, stream=s)
            l = ep.ep_router_logits(n.y, f.gate, stream=s)
            idx, w = ep.ep_route(l, 8, score="sigmoid", bias=f.bias, num_groups=4, topk_groups=2,
                                 scale=1.5, stream=s)
            dl = ep.ep_route_backward(w, l, idx, score="sigmoid", stream=s)
            dx, dw = ep.ep_router_logits_backward(dl, n.y, f.gate, stream=s)
            got.append((n, l, idx, w, dx, dw))
    torch.cuda.synchronize()
    for g, f, (n, l, idx, w, *_) in zip(got, (a, b), want):
        assert torch.equal(g[0].y, n.y) and torch.equal(g[0].scale, n.scale)
        assert torch.equal(g[1], l) and torch.equal(g[2], idx) and torch.equal(g[3], w)
        dl = ep.ep_route_backward(w, l, idx, score="sigmoid")
        dx, dw = ep.ep_router_logits_backward(dl, n.y, f.gate)
        assert torch.equal(g[4], dx) and torch.equal(g[5], dw)


def test_tensors_of_two_devices_and_streams_are_refused():
    x = torch.zeros(2, 128, dtype=torch.bfloat16).cuda()
    w = torch.ones(128)
    with pytest.raises(ValueError, match="GPU"):
        ep.ep_rms_norm(x, w)
    with pytest.raises(ValueError, match="GPU"):
        ep.ep_router_logits(x, x.cpu())
    with pytest.raises(ValueError, match="GPU"):
        ep.dispatch((x.to(FP8), torch.ones(2, 1)), torch.zeros(2, 1, dtype=torch.int64).cuda(),
                    torch.ones(2, 1).cuda(), num_local_experts=1, num_ranks=1, num_send=2)
