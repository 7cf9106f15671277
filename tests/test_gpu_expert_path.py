"""The expert-side calls as they are used: a training step through dispatch,
expert and combine with every gradient against autograd in 64 bits, a serving
layer against the dispatch path, and the calls in captured graphs, on several
streams and with buffers of the caller's."""

import numpy as np
import pytest
import torch

from tests.expert_helpers import BF16, FORMATS, bf16, check, f64, make_weights, moe_ref, topk
from tests.gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

import combine_ep_send_amd as ep  # noqa: E402

DEV = "cuda:0"


def dev_weights(t, fmt, group):
    q, s = t
    return q.to(DEV) if fmt == "bf16" else ep.W4Weights(q.to(DEV), s.to(DEV), fmt, group)


# ---------------------------------------------------------------------------
# training: dispatch, regroup, two products, activation with checkpoint,
# restore, combine; and back
# ---------------------------------------------------------------------------

def segments(offsets):
    o = offsets.tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(o[:-1], o[1:])) if b > a]


@pytest.mark.parametrize("T,K,P,El,H,I", [(24, 2, 2, 2, 128, 128), (40, 3, 4, 2, 256, 128)])
def test_training_step(T, K, P, El, H, I):
    rng = np.random.default_rng(T)
    E = P * El
    idx, w = topk(rng, T, K, E, unrouted=0.1)
    x, dout = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H)))
    w13, w2 = bf16(rng.standard_normal((E, 2 * I, H)) / H ** .5), bf16(
        rng.standard_normal((E, H, I)) / I ** .5)
    d = dict(x=x, dout=dout, w13=w13, w2=w2, idx=torch.from_numpy(idx), w=torch.from_numpy(w))
    d = {k: v.to(DEV) for k, v in d.items()}

    # forward: every slot gets its own expert row, weighted where it is combined
    cap = T * min(K, P)
    recv_x, recv_idx, recv_w, handle = ep.dispatch(d["x"], d["idx"], d["w"], num_local_experts=El,
                                                   num_ranks=P, num_send=cap)
    n = int(handle.send_counts.sum())
    recv_x, recv_idx, recv_w = recv_x[:n].contiguous(), recv_idx[:n].contiguous(), recv_w[:n]
    rg = ep.permute_by_expert(recv_x, recv_idx, recv_w.contiguous(), num_local_experts=El,
                              pad_multiple=8, row_group=handle.send_rank[:n], num_groups=P)
    rows = int(rg.expert_offsets[-1])
    px = rg.perm_x[:rows]
    gu = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device=DEV)
    for e, a, b in segments(rg.expert_offsets):
        gu[a:b] = px[a:b] @ d["w13"][e].t()
    h, q, scale = ep.ep_swiglu_fp8(gu, row_count=rg.expert_offsets[-1:])
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    for e, a, b in segments(rg.expert_offsets):
        y[a:b] = h[a:b] @ d["w2"][e].t()
    part = ep.restore_by_expert(y, rg, recv_w.contiguous())          # weighted partial rows
    buf = torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV)
    buf[:n] = part
    out = ep.combine(buf, handle, weighted=False)

    # backward
    dpart, none = ep.combine_backward(d["dout"], buf, handle, weighted=False)
    assert none is None and (dpart[n:] == 0).all()
    dy, dw_rows = ep.ep_combine_backward(dpart[:n].contiguous(), y, rg.row_map,
                                         recv_w.contiguous())
    pad = torch.ones(rows, dtype=torch.bool, device=DEV)
    pad[rg.perm_src[:rows] >= 0] = False
    assert (dy[pad] == 0).all()
    dh, dw2 = torch.zeros_like(h), torch.zeros_like(d["w2"])
    dgu_x, dw13 = torch.zeros_like(px), torch.zeros_like(d["w13"])
    for e, a, b in segments(rg.expert_offsets):
        dh[a:b] = dy[a:b] @ d["w2"][e]
    dgu, again = ep.ep_swiglu_fp8_backward(dh, q, scale, row_count=rg.expert_offsets[-1:])
    for e, a, b in segments(rg.expert_offsets):
        dw2[e] = dy[a:b].t() @ again[a:b]
        dw13[e] = dgu[a:b].t() @ px[a:b]
        dgu_x[a:b] = dgu[a:b] @ d["w13"][e]
    drecv = torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV)
    drecv[:n] = ep.ep_combine(dgu_x, rg.row_map, None)
    dx = ep.dispatch_backward(drecv, handle)
    dw = torch.zeros(T, K, device=DEV)
    # a slot's weight gradient sits at its send row's slot of the same number
    ok = handle.token_row >= 0
    dw[ok] = dw_rows[handle.token_row[ok].long(), ok.nonzero()[:, 1]]
    torch.cuda.synchronize()

    # the same in 64 bits, by autograd, through the same codes (the backward is
    # the gradient at the checkpoint's values, so the activations are replaced
    # by those values and the products before them keep their gradients)
    X, W, W13, W2 = (t.double().requires_grad_() for t in (x, d["w"].cpu(), w13, w2))
    kept = (q.float().cpu().double().view(rows, -1, 128) *
            scale.cpu().double()[..., None]).view(rows, 2 * I)
    src, slot_of = rg.perm_src.cpu(), rg.row_map.cpu()
    tok = handle.send_token_idx.cpu()
    total = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(handle.token_row[t, k])
            if r < 0:
                continue
            assert int(tok[r]) == t
            j = int(slot_of[r, k])
            e = int(idx[t, k])
            assert int(src[j]) == r
            exact = W13[e] @ X[t]
            v = exact + (kept[j] - exact).detach()
            hh = v[:I] * torch.sigmoid(v[:I]) * v[I:]
            total[t] += W[t, k] * (W2[e] @ hh)
    total.backward(dout.double())

    def near(got, ref, what):
        """At most 10 roundings to bf16 lie between the inputs and a gradient,
        each off by up to 2^-8 of a value, independent of the others and of the
        signs in the sums, which therefore grow errors and values alike: 12 *
        2^-8 in the 2-norm if every rounding were as bad as the worst."""
        got, ref = got.detach().cpu().double(), ref.detach()
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= 12 * BF16, (what, rel)
    # the forward used the activation itself, not its checkpoint: 8-bit codes
    # are off by 2^-4 relative at most, and so is the output
    rel = float((out.cpu().double() - total.detach()).norm() / total.detach().norm())
    assert rel <= 2 * 2.0 ** -4 + 12 * BF16, rel
    near(dx, X.grad, "dx")
    near(dw13, W13.grad, "dw13")
    near(dw2, W2.grad, "dw2")
    # the weights' gradient reads the forward's y, which the checkpoint does not enter
    rel = float((dw.cpu().double() - W.grad).norm() / W.grad.norm())
    assert rel <= 2 * 2.0 ** -4 + 12 * BF16, rel


# ---------------------------------------------------------------------------
# serving
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,group", FORMATS)
def test_layer_against_the_dispatch_path(fmt, group):
    """Two ranks' layers of a few tokens, added up, give what dispatch, the
    row products and combine give for all experts."""
    rng = np.random.default_rng(31)
    T, K, E, H, I = 6, 4, 8, 256, 128
    t13, v13, m13 = make_weights(rng, fmt, group, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, fmt, group, E, H, I)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, E, unrouted=0.1)
    d_x, d_idx, d_w = x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)
    w13, w2 = dev_weights(t13, fmt, group), dev_weights(t2, fmt, group)

    def part(wt, a, b):
        if fmt == "bf16":
            return wt[a:b]
        return ep.W4Weights(wt.q[a:b], wt.scale[a:b], fmt, group)
    low = ep.ep_moe_tokens(d_x, d_idx, d_w, part(w13, 0, 3), part(w2, 0, 3), 0)
    both = ep.ep_moe_tokens(d_x, d_idx, d_w, part(w13, 3, 8), part(w2, 3, 8), 3, bias=low)
    ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 0)
    first, _ = moe_ref(f64(x), np.where(idx < 3, idx, -1), w, v13, m13, v2, m2, 0)
    check(both, ref, tol + 1.01 * BF16 * np.abs(first), "two ranks")

    # every slot its own row: products, activation, products, combine
    slots = torch.arange(T * K, device=DEV).view(T, K).to(torch.int32)
    rows = torch.where(d_idx >= 0, slots, -1)
    ids = d_idx.reshape(-1).to(torch.int32)
    px = d_x.repeat_interleave(K, 0).contiguous()
    gu = ep.ep_expert_matvec(px, w13, ids)
    h, _, _ = ep.ep_swiglu_fp8(gu)
    y = ep.ep_expert_matvec(h, w2, ids)
    out = ep.ep_combine(y, rows, d_w)
    whole = ep.ep_moe_tokens(d_x, d_idx, d_w, w13, w2)
    check(whole, ref, tol, "layer")
    # the path rounds gate and up, h, y and out to bf16; the layer only out
    g, u = np.einsum("enh,th->ten", v13, f64(x))[:, :, :I], np.einsum("enh,th->ten", v13,
                                                                      f64(x))[:, :, I:]
    hh = np.abs(g / (1 + np.exp(-g)) * u)
    hmax = 1.1 * np.abs(g) * np.abs(u) * BF16 + 3 * BF16 * hh
    more = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            e = idx[t, k]
            if e >= 0:
                size = np.abs(v2[e]) @ hmax[t, e] + BF16 * (np.abs(v2[e]) @ hh[t, e])
                more[t] += w[t, k] * size
    check(out, ref, tol + 1.1 * more, "rows")


def test_replayed_graphs_share_nothing():
    """Two graphs of the layer captured on one stream and replayed on two at
    once, with eager calls between the replays: every output is the eager one."""
    rng = np.random.default_rng(41)
    K, E, H, I = 2, 6, 256, 128
    t13, _, _ = make_weights(rng, "fp4", 32, E, 2 * I, H)
    t2, _, _ = make_weights(rng, "fp4", 32, E, H, I)
    w13, w2 = dev_weights(t13, "fp4", 32), dev_weights(t2, "fp4", 32)
    cases = []
    for T in (3, 50):
        x = bf16(rng.standard_normal((T, H))).to(DEV)
        idx, w = (torch.from_numpy(a).to(DEV) for a in topk(rng, T, K, E))
        ep.ep_moe_tokens(x, idx, w, w13, w2)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ep.ep_moe_tokens(x, idx, w, w13, w2)
        cases.append((g, x, idx, w, out, torch.cuda.Stream()))
    for turn in range(4):
        for g, x, idx, w, out, s in cases:
            x.copy_(bf16(rng.standard_normal(tuple(x.shape))))
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, x, idx, w, out, s in cases:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for g, x, idx, w, out, s in cases:
            eager = ep.ep_moe_tokens(x, idx, w, w13, w2)
            assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), turn


def test_replayed_graph_of_the_training_calls():
    rng = np.random.default_rng(42)
    R, I, T, K, H = 20, 128, 10, 2, 256
    gu, dh = bf16(rng.standard_normal((R, 2 * I))).to(DEV), bf16(rng.standard_normal((R, I))).to(DEV)
    dout, y = bf16(rng.standard_normal((T, H))).to(DEV), bf16(rng.standard_normal((T * K, H))).to(DEV)
    row = torch.randperm(T * K, device=DEV).view(T, K).to(torch.int32)
    w = torch.rand(T, K, device=DEV)
    x, ids = bf16(rng.standard_normal((5, H))).to(DEV), torch.zeros(5, dtype=torch.int32, device=DEV)
    mat = bf16(rng.standard_normal((1, 64, H))).to(DEV)

    def run():
        h, q, s = ep.ep_swiglu_fp8(gu)
        d, again = ep.ep_swiglu_fp8_backward(dh, q, s)
        dy, dw = ep.ep_combine_backward(dout, y, row, w)
        q4 = ep.ep_quantize_w4(mat)
        return [h, d, again, dy, dw, ep.ep_expert_matvec(x, mat, ids),
                ep.ep_expert_matvec(x, q4, ids)]
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for turn in range(4):
        gu.copy_(bf16(rng.standard_normal((R, 2 * I))))
        dout.copy_(bf16(rng.standard_normal((T, H))))
        mat.copy_(bf16(rng.standard_normal((1, 64, H))))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), turn


def test_streams():
    """A stream that is given is where the call runs, and what it allocates
    belongs there."""
    rng = np.random.default_rng(43)
    T, K, E, H, I = 30, 3, 4, 256, 128
    t13, v13, m13 = make_weights(rng, "int4", 64, E, 2 * I, H)
    t2, v2, m2 = make_weights(rng, "int4", 64, E, H, I)
    w13, w2 = dev_weights(t13, "int4", 64), dev_weights(t2, "int4", 64)
    x = bf16(rng.standard_normal((T, H)))
    idx, w = topk(rng, T, K, E)
    ref, tol = moe_ref(f64(x), idx, w, v13, m13, v2, m2, 0)
    d_idx, d_w = torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV)
    host = x.pin_memory()
    outs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                d_x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
                torch.cuda._sleep(200000)                    # the copy comes late
                d_x.copy_(host, non_blocking=True)
            outs.append(ep.ep_moe_tokens(d_x, d_idx, d_w, w13, w2, stream=s))
    torch.cuda.synchronize()
    for out in outs:
        check(out, ref, tol)


def test_refusals_on_the_device():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2, 16, 256, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    idx, tw = torch.zeros(4, 2, dtype=torch.int64, device=DEV), torch.zeros(4, 2, device=DEV)
    w13 = torch.zeros(2, 64, 256, dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros(2, 256, 32, dtype=torch.bfloat16, device=DEV)
    q = ep.ep_quantize_w4(w)
    bad = [
        lambda: ep.ep_expert_matvec(x.float(), w, ids),
        lambda: ep.ep_expert_matvec(x[:, :128], w, ids),
        lambda: ep.ep_expert_matvec(x[:, ::2], w, ids),
        lambda: ep.ep_expert_matvec(x, w),
        lambda: ep.ep_expert_matvec(x, w[0], ids),
        lambda: ep.ep_expert_matvec(x, w, ids.long()),
        lambda: ep.ep_expert_matvec(x, w, ids[:3]),
        lambda: ep.ep_expert_matvec(x, w, ids.cpu()),
        lambda: ep.ep_expert_matvec(x, w, ids, out=x),
        lambda: ep.ep_expert_matvec(x, q._replace(group=64), ids),
        lambda: ep.ep_expert_matvec(x, q._replace(group=0), ids),
        lambda: ep.ep_expert_matvec(x, q._replace(fmt="fp4"), ids),
        lambda: ep.ep_expert_matvec(x, q._replace(fmt="int8"), ids),
        lambda: ep.ep_expert_matvec(x, q._replace(q=q.q.cpu()), ids),
        lambda: ep.ep_expert_matvec(x.new_zeros(1025, 256), w[:1]),
        lambda: ep.ep_expert_matvec(x.new_zeros(4 * 256 + 8)[4:-4].view(4, 256), w, ids),
        lambda: ep.ep_quantize_w4(w[..., :64].contiguous()),
        lambda: ep.ep_quantize_w4(w, "fp4", 64),
        lambda: ep.ep_moe_tokens(x, idx.int(), tw, w13, w2),
        lambda: ep.ep_moe_tokens(x, idx, tw.double(), w13, w2),
        lambda: ep.ep_moe_tokens(x, idx[:3], tw, w13, w2),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13[:, :32], w2),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2[:1]),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, -1),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, bias=[x, x, x]),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, bias=x[:2]),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, workspace=x.new_empty(64, dtype=torch.uint8)),
        lambda: ep.ep_moe_tokens(x.new_zeros(129, 256), idx.new_zeros(129, 2),
                                 tw.new_zeros(129, 2), w13, w2),
        lambda: ep.ep_swiglu_fp8(x[:, :128].contiguous()),
        lambda: ep.ep_swiglu_fp8(x, row_count=ids),
        lambda: ep.ep_swiglu_fp8(x, out=x),
        lambda: ep.ep_swiglu_fp8_backward(x, x, x),
        lambda: ep.ep_combine_backward(x, None, ids.view(2, 2), tw),
        lambda: ep.ep_combine_backward(x, x, ids.view(4, 1), tw),
        lambda: ep.ep_combine_backward(x, None, ids.view(4, 1), tw[:, :1].contiguous()),
        lambda: ep.ep_combine_backward(x, x[:, :128].contiguous(), ids.view(4, 1), None),
        lambda: ep.ep_combine_backward(x, x, ids.view(4, 1), None, dw=tw[:, :1].contiguous()),
        lambda: ep.ep_combine_backward(x, None, ids.view(4, 1), None),
        lambda: ep.ep_combine_backward(x, x, ids.view(4, 1), None, num_rows=5),
    ]
    big = 1 << 32                      # plus a size that would pass without it
    none = x.new_zeros(0, big + 256)
    bad += [
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, big),
        lambda: ep.ep_moe_tokens(x, idx, tw, w13, w2, -big),
        lambda: ep.ep_moe_tokens(x[:0], idx.new_zeros(0, big + 2), tw.new_zeros(0, big + 2), w13,
                                 w2),
        lambda: ep.ep_quantize_w4(w, "int4", big + 32),
        lambda: ep.ep_quantize_w4(w, "int4", 16),
        lambda: ep.ep_quantize_w4(none),
        lambda: ep.ep_expert_matvec(x, q._replace(group=big + 128), ids),
        lambda: ep.ep_expert_matvec(x[:, :0].contiguous(), x.new_zeros(1, big + 1, 0)),
        lambda: ep.ep_swiglu_fp8(x.new_zeros(0, 2 * big + 256)),
        lambda: ep.ep_swiglu_fp8_backward(none, none.new_zeros(0, 2 * (big + 256)),
                                          none.new_zeros(0, (big + 256) // 64)),
        lambda: ep.ep_combine_backward(none, none, ids.view(4, 1)[:0], None),
        lambda: ep.ep_combine_backward(x[:0], x, ids.new_zeros(0, big + 1), None),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted:", i, flush=True)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,K", [(1, 1), (4, 2), (20, 2), (40, 2), (70, 2)])
def test_layer_carries_h_within_two_to_the_minus_17(T, K):
    """One-hot rows make h = g * u of 24 bits exactly, an identity as the second
    matrix and minus bf16(h) as the bias leave what bf16 does not hold of h."""
    rng = np.random.default_rng(T)
    E, H, I = 2, 256, 256
    w13 = np.zeros((E, 2 * I, H))
    a, b, g = rng.integers(128, 256, (3, E, I))
    w13[:, :I, 0], w13[:, I:, 1], w13[:, I:, 2] = g, a, b      # exp(-128) adds nothing to 1
    h = g * (a + b * 2.0 ** -8)
    assert (h.astype(np.float32) == h).all()
    x = np.zeros((T, H))
    x[:, 0], x[:, 1], x[:, 2] = 1, 1, 2.0 ** -8
    idx = np.full((T, K), -1, np.int64)
    idx[:, 0] = rng.integers(0, E, T)
    w = np.ones((T, K), np.float32)
    near = f64(bf16(h))
    out = ep.ep_moe_tokens(bf16(x).to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV),
                           bf16(w13).to(DEV), bf16(np.broadcast_to(np.eye(H), (E, H, I))).to(DEV),
                           bias=bf16(-near[idx[:, 0]]).to(DEV))
    rest = (h - near)[idx[:, 0]]
    check(out, rest, 2.0 ** -17 * h[idx[:, 0]] + BF16 * np.abs(f64(out.cpu())))


def test_layer_keeps_h_finite_up_to_the_largest_number():
    """h of all 24 bits set just below 2^128, where rounding to bf16 overflows."""
    H = I = 128
    w13 = np.zeros((1, 2 * I, H))
    w13[0, :I, 0], w13[0, I:, 1], w13[0, I:, 2] = 128, 255, 255
    top = 128 * (255 + 255 * 2.0 ** -8)
    x = np.zeros((1, H))
    x[0, :3] = 1, 2.0 ** 113, 2.0 ** 105
    w2 = np.eye(H)[None] * 2.0 ** -60
    out = ep.ep_moe_tokens(bf16(x).to(DEV), torch.zeros(1, 1, dtype=torch.int64, device=DEV),
                           torch.ones(1, 1, device=DEV), bf16(w13).to(DEV), bf16(w2).to(DEV))
    ref = np.full((1, H), top * 2.0 ** 53)
    assert top * 2.0 ** 113 < 2.0 ** 128
    check(out, ref, (BF16 + 2.0 ** -15) * ref)
