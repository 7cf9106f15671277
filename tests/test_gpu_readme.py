"""README.md's Python examples run as they stand, one after the other, with the arrays
and the experts that a user brings; the training example's gradients are checked."""

import os
import re

import numpy as np
import pytest
import torch

from tests.router_forms import BF16, TINY, bf16, check, f64, logits_backward_ref

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def codes_to_bf16(rows, *_):
    q, scale = rows
    return (q.float().unflatten(-1, (-1, 128)) * scale[..., None]).flatten(-2).bfloat16()


def test_examples_run():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 3
    T, H, E, K, I = 40, 256, 256, 8, 128
    rng = np.random.default_rng(0)

    def rows(*shape, by=1.0):
        return bf16(by * rng.standard_normal(shape)).cuda()
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :K].copy()).cuda()
    have = dict(T=T, K=K, H=H, x=rows(T, H), topk_idx=idx, topk_weights=torch.rand(T, K).cuda(),
                expert=lambda recv, *_: recv, expert_fp8=codes_to_bf16)
    exec(blocks[0], have)
    assert have["out"].shape == (T, H) and have["out"].isfinite().all()

    # experts that differ, by powers of two: the router has a gradient then
    factor = 2.0 ** np.arange(-1, 3)[np.arange(32) % 4]

    def by():
        rank = have["handle"].send_rank.long() % 32
        return torch.from_numpy(factor).cuda()[rank, None].bfloat16()
    have.update(residual=rows(T, H), weight=torch.ones(H).cuda(), gate=rows(E, H, by=H ** -0.5),
                bias=torch.zeros(E).cuda(), d_out=rows(T, H),
                expert_fp8=lambda recv, *_: codes_to_bf16(recv) * by(),
                expert_backward=lambda d: d * by())
    exec(blocks[1], have)
    idx, w, d_out = have["topk_idx"].cpu().numpy(), f64(have["topk_weights"]), f64(have["d_out"])
    row = f64(have["handle"].token_row).astype(int)
    # the slots' weights: each a sum of H products in fp32
    y = f64(have["y"])[row]
    check(have["d_w"], np.einsum("th,tkh->tk", d_out, y),
          (H + 8) * 2.0 ** -24 * np.einsum("th,tkh->tk", np.abs(d_out), np.abs(y)) + TINY, "d_w")
    # both users of n.y; a destination's row once
    ref, tol, _, _ = logits_backward_ref(f64(have["d_logits"]), f64(have["n"].y),
                                         f64(have["gate"]))
    size = np.abs(ref)
    for r in range(32):
        part = factor[r] * (w * (idx // 8 == r)).sum(1, keepdims=True) * d_out
        ref, size = ref + part, size + np.abs(part)
    check(have["d_y"], ref, tol + 1.01 * BF16 * size + BF16 * np.abs(ref) + TINY, "d_y")
    assert np.abs(f64(have["d_logits"])).max() > 0.1

    have.update(x=have["x"][:3].contiguous(), topk_idx=have["topk_idx"][:3].contiguous(),
                topk_weights=have["topk_weights"][:3].contiguous(),
                gate_up_matrices=rows(E, 2 * I, H, by=0.1), down_matrices=rows(E, H, I, by=0.1),
                gate_up=rows(len(have["y"]), 2 * I), d_h=rows(len(have["y"]), I))
    exec(blocks[2], have)
    assert have["out"].shape == (3, H) and have["d_x"].shape == (T, H)
