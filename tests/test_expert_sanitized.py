"""Host-side validation of the expert-side calls under the address and
undefined-behaviour sanitizers (host code only), as test_abi_sanitized.py does
for the other header: tests/c/expert_sweep.cpp.  Runs only where there is no
GPU, since what passes validation reaches a launch on fake pointers."""

import os

import pytest

from tests.test_abi_sanitized import CSRC, HIPCC, ROOT, SAN, _run

pytestmark = [
    pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found"),
    pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="runs only where there is no GPU"),
]


def test_validation_is_clean_under_sanitizers(tmp_path):
    lib, exe = tmp_path / "libepdc_expert_san.so", tmp_path / "expert_sweep"
    inc = ["-I", os.path.join(ROOT, "include")]
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", "-shared",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *SAN, *inc,
          "-o", str(lib),
          *[os.path.join(CSRC, s) for s in ("expert.hip", "grad.hip", "expert_api.hip")]],
         timeout=900)
    _run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", *SAN, *inc, "-o", str(exe),
          os.path.join(ROOT, "tests", "c", "expert_sweep.cpp"), "-L", str(tmp_path),
          "-lepdc_expert_san", f"-Wl,-rpath,{tmp_path}"], timeout=300)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    for seed in ("1", "2"):
        out = _run([str(exe), seed, "700000"], timeout=300, env=env).stdout
        assert out.startswith("done:"), out
