"""The rules of the launches before the dispatch, as the library's own header has
them: host arithmetic, so no GPU is needed."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from combine_ep_send_amd import build
from tests.expert_forms import CSRC
from tests.router_forms import DEEP

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")

RULES = r"""
#include "router_rules.h"
using namespace epdc;
extern "C" int64_t live(int64_t T, int64_t count) { return route_live(T, count); }
extern "C" int64_t row(int64_t t, int64_t live) { return route_row(t, live); }
extern "C" int norm(int64_t T, int H, int* f) {
  f[0] = norm_shape(H).pieces, f[1] = norm_shape(H).threads;
  return norm_groups(T, H);
}
extern "C" void forms(int64_t T, int E, int H, int64_t* f) {
  const LogitsShape g = logits_shape(T, E, H);
  f[0] = g.wide, f[1] = g.bm, f[2] = g.wn, f[3] = g.nb, f[4] = g.each, f[5] = g.splits;
  const DxShape x = dx_shape(T, H, int(pad64(E)));
  f[6] = x.mt, f[7] = x.mb, f[8] = x.each;
  const DwShape w = dw_shape(T, E, H);
  f[9] = w.eb, f[10] = w.splits, f[11] = w.each;
}
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
    lib.norm.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.forms.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return lib


def test_every_product_is_tested_over_many_stages(rules):
    """DEEP reaches each form of the logits with more stages a workgroup than its ring of
    three and a turn that is not whole, each that splits the channels or not, and several
    workgroups of experts; the rows' gradient in each of its sizes over several workgroups
    and blocks of channels; the weights' in several parts and steps."""
    logits, split, experts, dx, dw = set(), set(), set(), set(), set()
    for T, E, H in DEEP:
        f = (ctypes.c_int64 * 12)()
        rules.forms(T, E, H, f)
        wide, bm, wn, nb, each, splits, mt, mb, dx_each, eb, dw_splits, dw_each = f
        form = "wide" if wide else (bm, wn)
        if each > 3 and each % 3:
            logits.add(form)
            split.add((form, splits > 1))
        if nb > 2 or (nb > 1 and not wide):
            experts.add(form)
        if T > 16 * mt and mb > 1 and dx_each > 4:
            dx.add(mt)
        dw.add((eb > 1, dw_splits > 1, dw_each > 4))
    assert logits == {(64, 1), (64, 2), (64, 4), (32, 4), (16, 4), "wide"}
    assert split >= {((64, 1), False), ((64, 2), False), ((64, 4), True), ((32, 4), True),
                     ((16, 4), True), ("wide", False), ("wide", True)}
    assert experts >= {(64, 4), (32, 4), (16, 4), "wide"}
    assert dx == {1, 2, 4}
    assert dw >= {(False, True, True), (True, True, True), (True, False, False)}


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


@pytest.mark.skipif(not os.path.exists(build.hipcc()), reason="hipcc not found")
def test_the_chip_holds_the_norms_backward_workgroups_at_once(rules, tmp_path):
    """The waves a compute unit that norm_groups counts on, by the registers of the kernels
    as the compiler reports them: as many workgroups as fit, four at most."""
    flags = [f for f in build.HIPCC_FLAGS if f != "-shared"]
    out = subprocess.run([build.hipcc(), *flags, "-I", os.path.join(build.ROOT, "include"),
                          "-Rpass-analysis=kernel-resource-usage", "--cuda-device-only", "-c", "-o",
                          str(tmp_path / "norm.o"), os.path.join(CSRC, "norm.hip")],
                         capture_output=True, text=True, check=True).stderr
    waves = {}
    for name, simd in re.findall(r"Function Name: (\S+).*?Occupancy \[waves/SIMD\]: (\d+)", out,
                                 re.S):
        m = re.search(r"rms_norm_backward_kernelILi(\d)E", name)
        if m:
            waves.setdefault(int(m.group(1)), set()).add(4 * int(simd))
    assert set(waves) == {1, 2, 4, 8} and all(len(v) == 1 for v in waves.values()), waves
    for H in (8, 520, 1032, 2056, 2560, 4096, 4104, 5120, 7168, 8192, 12288, 16384, 24576, 32768):
        f = (ctypes.c_int * 2)()
        each = rules.norm(1 << 29, H, f) // 256
        fit = next(iter(waves[f[0]])) // (f[1] // 64)
        assert each == max(1, min(4, fit)), (H, each, fit)
