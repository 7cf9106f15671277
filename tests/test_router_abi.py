"""The router-side header and its bindings agree, and every call refuses bad
arguments on the host, before it touches a GPU (none is needed here)."""

import ctypes
import os
import re

import pytest
import torch

import combine_ep_send_amd as ep
from combine_ep_send_amd import _lib
from tests.test_expert_abi import A16, A256, BAD, ODD4, ODD16, UNS, WS, call, refusals

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libepdc.so not built")

P = ctypes.c_void_p


def test_bindings_and_library_follow_the_header():
    assert set(_lib.header_functions(_lib.ROUTER_HEADER)) == set(_lib._ROUTER_SIGNATURES)
    text = open(_lib.ROUTER_HEADER).read()
    version = int(re.search(r"#define EPDC_ROUTER_ABI_VERSION (\d+)", text).group(1))
    assert version == _lib.ROUTER_ABI_VERSION == _lib.lib().ep_router_abi_version()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, (_, args) in _lib._ROUTER_SIGNATURES.items():
        params = re.search(name + r"\s*\(([^)]*)\)", code).group(1)
        n = 0 if params.strip() == "void" else params.count(",") + 1
        assert n == len(args), name
    for name in ("ep_rms_norm", "ep_rms_norm_backward", "ep_router_logits", "RmsNorm",
                 "ep_router_logits_backward", "ep_route", "ep_route_backward",
                 "ep_dispatch_permute_quantized"):
        assert hasattr(ep, name)


def test_norm_refusals():
    args = dict(x=A16, res=None, w=A16, wt=0, T=2, H=256, eps=1e-6, ro=None, out=A16, q=None,
                s=None, fmt=0, rstd=None, st=None)
    refusals(_lib.lib().ep_rms_norm, args, [
        (dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(H=0), BAD), (dict(H=-8), BAD),
        (dict(H=12), BAD), (dict(H=32776), UNS), (dict(wt=2), BAD), (dict(wt=-1), BAD),
        (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
        (dict(fmt=2), BAD), (dict(fmt=-1), BAD), (dict(x=None), BAD), (dict(x=ODD16), BAD),
        (dict(w=None), BAD), (dict(w=ODD16), BAD), (dict(res=A16), BAD), (dict(ro=A16), BAD),
        (dict(res=ODD16, ro=A16), BAD), (dict(res=A16, ro=ODD16), BAD), (dict(out=None), BAD),
        (dict(out=ODD16), BAD), (dict(q=A16), BAD), (dict(s=A16), BAD),
        (dict(q=ODD16, s=A16), BAD), (dict(q=A16, s=ODD4), BAD),
        (dict(q=A16, s=A16, H=264), BAD), (dict(rstd=ODD4), BAD),
        (dict(T=0, x=None, out=None), 0)])


def test_norm_backward_refusals():
    L = _lib.lib()
    size = L.ep_rms_norm_backward_workspace_bytes
    args = dict(dy=A16, s=A16, w=A16, wt=1, rstd=A16, dr=None, T=2, H=256, dx=A16, dw=A16, ws=A256,
                bytes=1 << 20, st=None)
    refusals(L.ep_rms_norm_backward, args, [
        (dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(H=0), BAD), (dict(H=12), BAD),
        (dict(H=1 << 16), UNS), (dict(wt=2), BAD), (dict(dy=None), BAD), (dict(dy=ODD16), BAD),
        (dict(s=None), BAD), (dict(s=ODD16), BAD), (dict(w=None), BAD), (dict(rstd=None), BAD),
        (dict(rstd=ODD4), BAD), (dict(dr=ODD16), BAD), (dict(dx=None), BAD), (dict(dx=ODD16), BAD),
        (dict(dw=ODD4), BAD), (dict(ws=None), WS), (dict(ws=A16), WS),
        (dict(bytes=size(2, 256) - 1), WS),
        (dict(T=0, dy=None, s=None, rstd=None, dx=None, dw=None, ws=None, bytes=0), 0)])
    assert size(2, 256) == 256 * 4 and size(64, 256) == 32 * 256 * 4
    assert size(0, 256) > 0
    for bad in ((-1, 256), (1 << 30, 256), (2, 0), (2, 12), (2, 32776), ((1 << 63) - 1, 256)):
        assert size(*bad) == 0


def test_logits_refusals():
    L = _lib.lib()
    size, back = L.ep_router_logits_workspace_bytes, L.ep_router_logits_backward_workspace_bytes
    both = [(dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(E=0), BAD), (dict(E=-3), BAD),
            (dict(E=1025), UNS), (dict(H=0), BAD), (dict(H=12), BAD), (dict(H=65544), UNS),
            (dict(ws=None), WS), (dict(ws=A16), WS)]
    refusals(L.ep_router_logits,
             dict(x=A16, w=A16, T=4, E=8, H=256, out=A16, ws=A256, bytes=1 << 24, st=None), both + [
                 (dict(x=None), BAD), (dict(x=ODD16), BAD), (dict(w=None), BAD),
                 (dict(w=ODD16), BAD), (dict(out=None), BAD), (dict(out=ODD4), BAD),
                 (dict(bytes=size(4, 8, 256) - 1), WS), (dict(T=0, x=None, out=None), 0)])
    refusals(L.ep_router_logits_backward,
             dict(d=A16, x=A16, w=A16, T=4, E=8, H=256, dx=A16, dw=A16, ws=A256, bytes=1 << 24,
                  st=None), both + [
                 (dict(d=None), BAD), (dict(d=ODD4), BAD), (dict(x=None), BAD),
                 (dict(x=ODD16), BAD), (dict(w=None), BAD), (dict(w=ODD16), BAD),
                 (dict(dx=ODD16), BAD), (dict(dw=ODD16), BAD), (dict(dx=None, dw=None), BAD),
                 (dict(bytes=back(4, 8, 256) - 1), WS),
                 (dict(T=0, d=None, x=None, dx=None, dw=None), 0)])
    for bad in ((-1, 8, 256), (1 << 30, 8, 256), (4, 0, 256), (4, 1025, 256), (4, 8, 12),
                (4, 8, 65544), ((1 << 63) - 1, 8, 256)):
        assert size(*bad) == back(*bad) == 0
    assert ep.ep_router_logits_workspace_bytes(4, (1 << 32) + 8, 256) == 0
    assert ep.ep_router_logits_backward_workspace_bytes((1 << 64) + 4, 8, 256) == 0


def test_route_refusals():
    L = _lib.lib()
    nan, inf = float("nan"), float("inf")
    both = [(dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(E=0), BAD), (dict(E=1025), UNS),
            (dict(K=0), BAD), (dict(K=17), UNS), (dict(score=2), BAD), (dict(score=-1), BAD),
            (dict(scale=nan), BAD), (dict(scale=inf), BAD)]
    refusals(L.ep_route,
             dict(l=A16, T=4, E=8, K=2, score=0, bias=None, G=1, kept=1, top=1, renorm=1, scale=1.0,
                  count=None, idx=A16, w=A16, st=None), both + [
                 (dict(G=0), BAD), (dict(G=3), BAD), (dict(kept=0), BAD), (dict(kept=2), BAD),
                 (dict(top=0), BAD), (dict(top=3), BAD), (dict(G=32, E=64), UNS),
                 (dict(l=None), BAD), (dict(l=ODD4), BAD), (dict(bias=ODD4), BAD),
                 (dict(count=ODD4), BAD), (dict(idx=None), BAD), (dict(idx=P(0x10004)), BAD),
                 (dict(w=None), BAD), (dict(w=ODD4), BAD), (dict(T=0, l=None, idx=None, w=None), 0)])
    refusals(L.ep_route_backward,
             dict(dw=A16, l=A16, idx=A16, T=4, E=8, K=2, score=1, renorm=1, scale=1.0, out=A16,
                  st=None), both + [
                 (dict(dw=None), BAD), (dict(dw=ODD4), BAD), (dict(l=None), BAD),
                 (dict(idx=None), BAD), (dict(idx=P(0x10004)), BAD), (dict(out=None), BAD),
                 (dict(out=ODD4), BAD), (dict(T=0, dw=None, l=None, idx=None, out=None), 0)])


def test_quantized_permute_refusals():
    refusals(_lib.lib().ep_dispatch_permute_quantized,
             dict(q=A16, s=A16, words=2, T=4, H=256, row=A16, K=2, cap=8, sq=A16, ss=A16, st=None), [
                 (dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(H=0), BAD), (dict(H=64), BAD),
                 (dict(H=1 << 27), UNS), (dict(words=-1), BAD), (dict(words=1 << 27), UNS),
                 (dict(K=0), BAD), (dict(K=17), UNS), (dict(cap=-1), BAD), (dict(cap=1 << 31), UNS),
                 (dict(q=None), BAD), (dict(q=ODD16), BAD), (dict(s=None), BAD), (dict(s=ODD4), BAD),
                 (dict(row=None), BAD), (dict(row=ODD4), BAD), (dict(sq=None), BAD),
                 (dict(sq=ODD16), BAD), (dict(ss=None), BAD), (dict(ss=ODD4), BAD),
                 (dict(T=0, q=None, s=None, row=None), 0), (dict(cap=0, sq=None, ss=None), 0)])


def test_python_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    w = torch.zeros(128, dtype=torch.bfloat16)
    f = torch.zeros(2, 128)
    idx = torch.zeros(2, 1, dtype=torch.int64)
    q = x.to(torch.float8_e4m3fn)
    for call_ in (lambda: ep.ep_rms_norm(x, w), lambda: ep.ep_rms_norm_backward(x, x, w, f),
                  lambda: ep.ep_router_logits(x, x),
                  lambda: ep.ep_router_logits_backward(f, x, x), lambda: ep.ep_route(f, 2),
                  lambda: ep.ep_route_backward(f, f, idx),
                  lambda: ep.ep_dispatch_permute_quantized(q, f, idx.int(), 2)):
        with pytest.raises(ValueError, match="GPU"):
            call_()
    with pytest.raises(TypeError):
        ep.ep_rms_norm(None, w)
    assert call(_lib.lib().ep_router_abi_version, {}) == 1
