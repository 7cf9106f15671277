"""Every product kernel of the few-row calls against exact outputs, to the bit."""

import pytest
import torch

from tests import expert_forms as F
from tests.gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

import combine_ep_send_amd as ep  # noqa: E402

DEV = "cuda:0"


def on_device(t, kind):
    fmt, group = F.KINDS[kind]
    q = t[0].to(DEV)
    return q if fmt == "bf16" else ep.W4Weights(q, t[1].to(DEV), fmt, group)


def same(got, exact):
    want = exact.float().to(torch.bfloat16) + 0.0          # no negative zeros
    bad = got.view(torch.int16) != want.view(torch.int16)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("call,kind,sizes", list(F.cases()),
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_exact(call, kind, sizes):
    if call == "rows":
        t, v, x, ids = F.rows_inputs(kind, sizes)
        x, ids = x.to(DEV), ids.to(DEV)
        w = on_device(t, kind)
        got = ep.ep_expert_matvec(x, w, ids)
        again = ep.ep_expert_matvec(x, w, ids)
        exact = F.rows_exact(v, x, ids)
    else:
        t13, v13, t2, v2, x, idx, tw = F.layer_inputs(kind, sizes)
        x, idx, tw = x.to(DEV), idx.to(DEV), tw.to(DEV)
        w13, w2 = on_device(t13, kind), on_device(t2, kind)
        got = ep.ep_moe_tokens(x, idx, tw, w13, w2)
        again = ep.ep_moe_tokens(x, idx, tw, w13, w2)
        exact = F.layer_exact(v13, v2, x, idx, tw)
    same(got, exact)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("R", [3, 20])
@pytest.mark.parametrize("kind", ["bf16", "fp4", "int4g32", "int4g64", "int4g128"])
def test_subnormal_rows(kind, R):
    """Channels below 2^-126 times weights of 2^20 and so on: nothing is flushed."""
    fmt, group = F.KINDS[kind]
    N, K = 32, 256
    code = torch.arange(N, dtype=torch.uint8) % 16
    if fmt == "bf16":
        val = code.double() - 8
        w = (val * 2.0 ** 20)[:, None].expand(N, K).to(torch.bfloat16)[None].contiguous().to(DEV)
    else:
        e2m1 = torch.tensor(F.E2M1).double()
        val = code.double() - 8 if fmt == "int4" else \
            torch.where(code > 7, -1.0, 1.0) * e2m1[(code & 7).long()]
        q = (code | code << 4)[:, None].expand(N, K // 2)[None].contiguous().to(DEV)
        scale = torch.full((1, N, K // group), 2.0 ** 20, dtype=torch.bfloat16) if fmt == "int4" else \
            torch.full((1, N, K // group), 147, dtype=torch.uint8)
        w = ep.W4Weights(q, scale.to(DEV), fmt, group)
    x = torch.zeros(R, K, dtype=torch.bfloat16)
    tiny = [2.0 ** -133, -1.5 * 2.0 ** -130, 2.0 ** -127]
    for r in range(R):
        x[r, r * 13 % K] = tiny[r % 3]
    y = ep.ep_expert_matvec(x.to(DEV), w)
    same(y, (x.double().sum(1)[:, None] * val[None] * 2.0 ** 20).to(DEV))
