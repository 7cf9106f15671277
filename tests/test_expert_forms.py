"""The cases of tests/expert_forms.py take every product kernel the library has:
by the rules that choose a kernel, and by the kernels in the built library."""

import os
import re
import shutil
import subprocess

import pytest

from combine_ep_send_amd import _lib
from tests import expert_forms as F

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

WEIGHT_KIND = {0: "bf16", 1: "fp4", 2: "int4g32", 3: "int4g64", 4: "int4g128", 5: "stream"}


def test_every_kernel_has_a_case(tmp_path):
    lib = F.rules(str(tmp_path))
    reached = set()
    for call, kind, sizes in F.cases():
        took = F.kernels(lib, call, kind, sizes)
        assert all(k[1] == kind for k in took), (call, kind, sizes, took)
        reached.update(took)
    assert reached == set(F.every_kernel())
    assert len(reached) == 124


@pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH) or shutil.which("nm") is None,
                    reason="needs libepdc.so and nm")
def test_the_library_has_no_other_product_kernel():
    names = subprocess.run(["nm", "-C", _lib.LIB_PATH], capture_output=True, text=True,
                           check=True).stdout
    built = set()
    for form, args in re.findall(r"__device_stub__few_(thin|wide|down)_kernel<([^>]*)>", names):
        p = [int(a) for a in args.split(",")]
        kind = WEIGHT_KIND[p[0]]
        if form == "thin":                       # KIND, NT, NV, W, OUT, D
            built.add(("thin", kind, F.OUTS[p[4]], p[3]))
        elif form == "wide":                     # KIND, NT, NV, MT, XP, OUT, D
            built.add(("wide", kind, F.OUTS[p[5]], p[1], p[3]))
        else:                                    # KIND, NT, NV, D
            built.add(("down", kind, p[1]))
    assert built == set(F.every_kernel())


def test_inputs_are_exact_in_fp32():
    """Small cases on the CPU; the larger ones assert the same where they run."""
    for call, kind, sizes in F.cases():
        if kind == "stream":
            continue
        if call == "rows":
            t, v, x, ids = F.rows_inputs(kind, sizes)
            y = F.rows_exact(v, x, ids)
        else:
            t13, v13, t2, v2, x, idx, w = F.layer_inputs(kind, sizes)
            y = F.layer_exact(v13, v2, x, idx, w)
        assert (y == y.round()).all() and (y != 0).any()
