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
