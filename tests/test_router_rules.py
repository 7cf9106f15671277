"""The rules of the launches before the dispatch, as the library's own header has
them: host arithmetic, so no GPU is needed."""

import ctypes
import os
import shutil
import subprocess

import pytest

from tests.expert_forms import CSRC

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")

RULES = r"""
#include "router_rules.h"
using namespace epdc;
extern "C" int64_t live(int64_t T, int64_t count) { return route_live(T, count); }
extern "C" int64_t row(int64_t t, int64_t live) { return route_row(t, live); }
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    folder = tmp_path_factory.mktemp("rules")
    src, out = os.path.join(folder, "rules.cpp"), os.path.join(folder, "rules.so")
    with open(src, "w") as f:
        f.write(RULES)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-I", CSRC, "-o", out,
                    src], check=True)
    lib = ctypes.CDLL(out)
    for name in ("live", "row"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64]
    return lib


@pytest.mark.parametrize("tokens", [4, 16])
def test_no_logits_of_padding_are_read(rules, tokens):
    """Workgroups of 4 or 16 tokens, none of them past the last live one's: a token's
    own logits, or in the place of one that is padding or past the end a live one's."""
    for T in (1, 3, 16, 17, 63, 64):
        for count in (-(1 << 31), -1, 0, 1, 2, 15, 16, 17, 40, T, T + 1, (1 << 31) - 1):
            live = rules.live(T, count)
            assert live == min(T, max(0, count))
            for t0 in range(0, T, tokens):
                if t0 >= live:
                    continue                         # such a workgroup reads none
                for t in range(t0, t0 + tokens):
                    assert rules.row(t, live) == (t if t < live else live - 1)
