"""int4 products beside large channels: rows of one sign up to the documented
limit, a large or infinite channel under a zero weight, and what an infinite
channel gives, for the rows, the layer's first products and its second."""

import numpy as np
import pytest
import torch

from tests.expert_helpers import bf16, check, f64, make_weights, matvec_ref, topk
from tests.gpu_helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

import combine_ep_send_amd as ep  # noqa: E402

DEV = "cuda:0"
GROUPS = [32, 64, 128]
ROWS = [1, 3, 7, 40, 100]         # few rows a wave alone, and one to three row tiles


def w4(q, s, group):
    return ep.W4Weights(torch.as_tensor(q).to(DEV), s.to(DEV), "int4", group)


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("R", ROWS)
@pytest.mark.parametrize("group", GROUPS)
def test_rows_of_one_sign_up_to_the_limit(group, R):
    """Every channel just below 2^122: a group's sum of (code - 8) / 16 times x
    stays below 128 * 0.5 * 2^122 = 2^128 however the codes are signed."""
    rng = np.random.default_rng(group + R)
    N, K = 48, 512
    q = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    q[0, 0], q[0, 1], q[0, 2] = 0x00, 0xFF, 0x88          # all -8, all 7, all 0
    s = bf16(rng.uniform(0.5, 1.5, (1, N, K // group)) * 2.0 ** -20)
    c = np.stack([q & 15, q >> 4], -1).reshape(1, N, K).astype(np.float64) - 8
    v = c * np.repeat(f64(s), group, -1)
    x = bf16(np.full((R, K), 2.0 ** 122 * (1 - 2.0 ** -8)) * np.where(np.arange(R) % 2, -1, 1)[:, None])
    assert torch.isfinite(x).all() and float(x.abs().max()) < 2.0 ** 122
    ids = np.zeros(R, np.int32)
    ref, tol = matvec_ref(f64(x), ids, v, np.abs(v))
    y = ep.ep_expert_matvec(x.to(DEV), w4(q, s, group))
    check(y, ref, tol)
    assert (bits(y[:, 2]) == 0).all()


@pytest.mark.parametrize("big", [2.0 ** 24, 2.0 ** 60, 2.0 ** 121, -2.0 ** 121])
@pytest.mark.parametrize("R", ROWS)
@pytest.mark.parametrize("group", GROUPS)
def test_a_zero_weight_drops_its_channel(group, R, big):
    """The bits of a row do not depend on a channel whose weights are all zero."""
    rng = np.random.default_rng(R)
    E, N, K = 2, 40, 384
    (q, s), v, mag = make_weights(rng, "int4", group, E, N, K)
    at = [0, 131, 383]                                    # both halves of a byte
    codes = np.stack([q & 15, q >> 4], -1).reshape(E, N, K)
    codes[:, :, at] = 8
    q = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
    x = bf16(rng.standard_normal((R, K)))
    ids = torch.from_numpy(rng.integers(0, E, R).astype(np.int32)).to(DEV)
    x[:, at] = 0
    without = ep.ep_expert_matvec(x.to(DEV), w4(q, s, group), ids)
    x[:, at] = big
    beside = ep.ep_expert_matvec(x.to(DEV), w4(q, s, group), ids)
    assert torch.equal(bits(without), bits(beside))
    assert torch.isfinite(beside).all() and (beside != 0).any()


@pytest.mark.parametrize("T,K", [(2, 2), (9, 4), (60, 8)])     # joined; thin and wide apart
@pytest.mark.parametrize("group", GROUPS)
def test_layer_beside_large_channels(group, T, K):
    """A large channel of x under zero weights, and a large channel of h under
    zero weights, leave the layer's bits as they are."""
    rng = np.random.default_rng(T)
    E, H, I = 4, 256, 128
    (q13, s13), _, _ = make_weights(rng, "int4", group, E, 2 * I, H)
    (q2, s2), _, _ = make_weights(rng, "int4", group, E, H, I)
    q13, q2 = np.asarray(q13).copy(), np.asarray(q2).copy()
    q13[:, :, 5] = q13[:, :, 5] & 0xF0 | 8                # channel 10 of x
    q2[:, :, 20] = q2[:, :, 20] & 0x0F | 0x80             # channel 41 of h
    q13[:, [41, I + 41]] = 0xFF                           # its gate and up rows: all 7
    q13[:, [41, I + 41], 5] = 0xF8
    x = bf16(np.abs(rng.standard_normal((T, H))))
    x[:, 10] = 0
    idx, w = (torch.from_numpy(a).to(DEV) for a in topk(rng, T, K, E))

    def run(x, s13):
        return ep.ep_moe_tokens(x.to(DEV), idx, w, w4(q13, s13, group), w4(q2, s2, group))
    plain = run(x, s13)
    assert torch.isfinite(plain).all() and (plain != 0).any()
    x[:, 10] = 2.0 ** 121
    assert torch.equal(bits(run(x, s13)), bits(plain))
    s13[:, [41, I + 41]] = 2.0 ** 40                      # h[41] of 2^90 or so
    assert torch.equal(bits(run(x, s13)), bits(plain))


@pytest.mark.parametrize("R", ROWS)
@pytest.mark.parametrize("group", GROUPS)
def test_an_infinite_channel_gives_what_the_sum_gives(group, R):
    """Infinities of the weights' signs, NaN under a zero weight; the other
    rows are untouched."""
    rng = np.random.default_rng(R + 1)
    N, K = 32, 256
    (q, s), v, mag = make_weights(rng, "int4", group, 1, N, K)
    q = np.asarray(q).copy()
    q[0, :, 3] = np.arange(N) % 16 << 4 | q[0, :, 3] & 15     # channel 7: every code
    x = bf16(rng.standard_normal((R, K)))
    x[0, 7] = float("inf")
    y = ep.ep_expert_matvec(x.to(DEV), w4(q, s, group)).float().cpu().numpy()
    code = np.arange(N) % 16
    want = np.where(code == 8, np.nan, np.where(code > 8, np.inf, -np.inf))
    assert np.array_equal(y[0], want.astype(np.float32), equal_nan=True)
    assert np.isfinite(y[1:]).all()
