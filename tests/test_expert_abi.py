"""The expert-side header and its bindings agree, and every call refuses bad
arguments on the host, before it touches a GPU (none is needed here)."""

import ctypes
import os
import re

import pytest
import torch

import combine_ep_send_amd as ep
from combine_ep_send_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libepdc.so not built")

P = ctypes.c_void_p
A16, ODD16, ODD4, A256 = P(0x10010), P(0x10008), P(0x10002), P(0x10100)
BAD, UNS, WS = _lib.EP_ERR_INVALID_ARG, _lib.EP_ERR_UNSUPPORTED, _lib.EP_ERR_WORKSPACE
INT4, FP4, BF = _lib.EP_W_INT4, _lib.EP_W_FP4, _lib.EP_W_BF16


def test_bindings_and_library_follow_the_header():
    assert set(_lib.header_functions(_lib.EXPERT_HEADER)) == set(_lib._EXPERT_SIGNATURES)
    text = open(_lib.EXPERT_HEADER).read()
    version = int(re.search(r"#define EPDC_EXPERT_ABI_VERSION (\d+)", text).group(1))
    assert version == _lib.EXPERT_ABI_VERSION == _lib.lib().ep_expert_abi_version()
    # every declaration has as many parameters as its binding
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, (_, args) in _lib._EXPERT_SIGNATURES.items():
        params = re.search(name + r"\s*\(([^)]*)\)", code).group(1)
        n = 0 if params.strip() == "void" else params.count(",") + 1
        assert n == len(args), name
    for name in ("ep_moe_tokens", "ep_expert_matvec", "ep_quantize_w4", "ep_swiglu_fp8",
                 "ep_swiglu_fp8_backward", "ep_combine_backward", "combine_backward",
                 "dispatch_backward", "W4Weights"):
        assert hasattr(ep, name)


def call(fn, args, **change):
    return fn(*{**args, **change}.values())


def refusals(fn, args, cases):
    for change, status in cases:
        assert call(fn, args, **change) == status, (change, status)


def test_matvec_refusals():
    args = dict(x=A16, ids=A16, rows=4, E=2, N=64, K=128, fmt=INT4, group=64, w=A16, s=A16, y=A16,
                stream=None)
    refusals(_lib.lib().ep_expert_matvec, args, [
        (dict(rows=-1), BAD), (dict(rows=1025), UNS), (dict(rows=1 << 40), UNS),
        (dict(E=0), BAD), (dict(E=1025), UNS), (dict(N=0), BAD), (dict(N=-8), BAD),
        (dict(N=12), BAD), (dict(K=0), BAD), (dict(K=64), BAD), (dict(K=192), BAD),
        (dict(K=131072), UNS), (dict(N=65544), UNS), (dict(fmt=3), BAD), (dict(fmt=-1), BAD),
        (dict(group=0), BAD), (dict(group=16), BAD), (dict(group=256), BAD),
        (dict(fmt=FP4, group=64), BAD), (dict(fmt=BF, group=64), BAD), (dict(K=12, fmt=BF, group=0), BAD),
        (dict(N=65536, K=65536, fmt=BF, group=0), UNS), (dict(x=None), BAD), (dict(x=ODD16), BAD),
        (dict(ids=None), BAD), (dict(ids=ODD4), BAD), (dict(w=None), BAD), (dict(w=ODD16), BAD),
        (dict(s=None), BAD), (dict(s=ODD16), BAD), (dict(y=None), BAD), (dict(y=ODD16), BAD),
        (dict(rows=0), 0), (dict(rows=0, x=None, ids=None, y=None), 0)])


def test_layer_refusals():
    args = dict(x=A16, idx=A16, tw=A16, T=4, K=2, H=256, I=128, first=0, E=4, f13=INT4, g13=128,
                w13=A16, s13=A16, f2=FP4, g2=32, w2=A16, s2=A16, b0=None, b1=None, out=A16,
                ws=A256, bytes=1 << 24, stream=None)
    refusals(_lib.lib().ep_moe_tokens, args, [
        (dict(T=-1), BAD), (dict(T=129), UNS), (dict(K=0), BAD), (dict(K=17), UNS),
        (dict(T=128, K=9), UNS), (dict(E=0), BAD), (dict(E=1025), UNS), (dict(first=-1), BAD),
        (dict(H=0), BAD), (dict(I=0), BAD), (dict(I=-128), BAD), (dict(H=128 + 64), BAD),
        (dict(I=64), BAD), (dict(f2=BF, g2=0, I=12), BAD), (dict(f13=BF, g13=0, H=12), BAD),
        (dict(I=2 ** 31 - 1), UNS), (dict(H=2 ** 31 - 1), UNS), (dict(H=1 << 17), UNS),
        (dict(g13=32, s13=None), BAD), (dict(g13=0), BAD), (dict(g2=64), BAD), (dict(f2=7), BAD),
        (dict(x=None), BAD), (dict(x=ODD16), BAD), (dict(idx=None), BAD), (dict(idx=P(0x10004)), BAD),
        (dict(tw=None), BAD), (dict(tw=ODD4), BAD), (dict(out=None), BAD), (dict(out=ODD16), BAD),
        (dict(b0=ODD16), BAD), (dict(b1=ODD4), BAD), (dict(w13=None), BAD), (dict(w2=ODD16), BAD),
        (dict(s2=None), BAD), (dict(ws=None), WS), (dict(ws=A16), WS), (dict(bytes=1000), WS),
        (dict(T=0, x=None, idx=None, tw=None, out=None), 0)])
    size = _lib.lib().ep_moe_tokens_workspace_bytes
    assert size(4, 2, 256, 128) == size(0, 2, 256, 128) + 8 * 128 * 4
    assert call(_lib.lib().ep_moe_tokens, args, bytes=size(4, 2, 256, 128) - 1) == WS
    for bad in ((-1, 2, 256, 128), (4, 0, 256, 128), (4, 2, 0, 128), (4, 2, 256, 0),
                (129, 1, 256, 128), (128, 9, 256, 128), (4, 17, 256, 128), (4, 2, 256, 65537),
                (4, 2, 65537, 128), (1 << 62, 2, 256, 128)):
        assert size(*bad) == 0


def test_row_call_refusals():
    L = _lib.lib()
    refusals(L.ep_quantize_w4, dict(w=A16, rows=2, K=128, fmt=INT4, g=32, q=A16, s=A16, st=None), [
        (dict(rows=-1), BAD), (dict(rows=1 << 30), UNS), (dict(K=0), BAD), (dict(K=64), BAD),
        (dict(K=1 << 27), UNS), (dict(fmt=BF), BAD), (dict(g=8), BAD), (dict(fmt=FP4, g=128), BAD),
        (dict(w=None), BAD), (dict(q=ODD16), BAD), (dict(s=ODD16), BAD), (dict(rows=0, w=None), 0)])
    refusals(L.ep_swiglu_fp8, dict(gu=A16, rows=2, I=128, n=None, h=A16, q=A16, s=A16, st=None), [
        (dict(rows=-1), BAD), (dict(rows=1 << 30), UNS), (dict(I=0), BAD), (dict(I=64), BAD),
        (dict(I=1 << 27), UNS), (dict(gu=ODD16), BAD), (dict(n=ODD4), BAD), (dict(h=None), BAD),
        (dict(q=ODD16), BAD), (dict(s=None), BAD), (dict(s=ODD4), BAD), (dict(rows=0, gu=None), 0)])
    refusals(L.ep_swiglu_fp8_backward,
             dict(dh=A16, q=A16, s=A16, rows=2, I=128, n=None, d=A16, h=None, st=None), [
                 (dict(rows=-1), BAD), (dict(I=192), BAD), (dict(dh=None), BAD),
                 (dict(q=ODD16), BAD), (dict(s=ODD4), BAD), (dict(d=None), BAD),
                 (dict(h=ODD16), BAD), (dict(n=ODD4), BAD), (dict(rows=0, dh=None, d=None), 0)])
    refusals(L.ep_combine_backward,
             dict(dout=A16, y=A16, R=4, row=A16, w=A16, T=2, K=2, H=64, dy=A16, dw=A16, st=None), [
                 (dict(T=-1), BAD), (dict(T=1 << 30), UNS), (dict(K=0), BAD), (dict(K=17), UNS),
                 (dict(R=-1), BAD), (dict(R=1 << 31), UNS), (dict(H=0), BAD), (dict(H=12), BAD),
                 (dict(dout=None), BAD), (dict(y=None), BAD), (dict(y=ODD16), BAD),
                 (dict(row=None), BAD), (dict(w=None), BAD), (dict(w=ODD4), BAD),
                 (dict(dw=ODD4), BAD), (dict(dy=None), BAD), (dict(dy=ODD16), BAD),
                 (dict(T=0, dout=None, row=None), 0)])


def test_python_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    w = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    idx, tw = torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2, 1)
    row = torch.zeros(2, 1, dtype=torch.int32)
    for call_ in (lambda: ep.ep_expert_matvec(x, w), lambda: ep.ep_quantize_w4(w),
                  lambda: ep.ep_moe_tokens(x, idx, tw, w, w), lambda: ep.ep_swiglu_fp8(x),
                  lambda: ep.ep_swiglu_fp8_backward(x, x, x),
                  lambda: ep.ep_combine_backward(x, x, row, tw)):
        with pytest.raises(ValueError, match="GPU"):
            call_()
    with pytest.raises(TypeError):
        ep.ep_expert_matvec(None, w)
    assert ep.ep_moe_tokens_workspace_bytes((1 << 32) + 4, 2, 256, 128) == 0
    assert ep.ep_moe_tokens_workspace_bytes(4, (1 << 32) + 2, 256, 128) == 0
    with pytest.raises(ValueError, match="fmt"):
        ep.ep_quantize_w4(w, "int8")


def test_no_workspace_size_for_a_layer_that_is_refused():
    """The size is 0 exactly where the call refuses the sizes in every format."""
    L = _lib.lib()
    size, layer = L.ep_moe_tokens_workspace_bytes, L.ep_moe_tokens

    def refused(T, K, H, I):
        """By every pair of formats, before the workspace is looked at."""
        for f13, g13 in ((BF, 0), (INT4, 32), (FP4, 32)):
            for f2, g2 in ((BF, 0), (INT4, 32), (FP4, 32)):
                st = layer(A16, A16, A16, T, K, H, I, 0, 4, f13, g13, A16, A16, f2, g2, A16, A16,
                           None, None, A16, None, 0, None)
                assert st in (BAD, UNS, WS)
                if st == WS:
                    return False
        return True
    for H in (8, 12, 100, 104, 128, 7168, 32768, 65528, 65536, 65544):
        for I in (4, 8, 12, 128, 200, 2048, 32760, 32768, 65535, 65536):
            for T, K in ((1, 1), (128, 8)):
                assert (size(T, K, H, I) == 0) == refused(T, K, H, I), (T, K, H, I)
