"""The rule that cuts norm and rotation into workgroups, swept on the CPU over
head dimensions, rotated pairs, layouts, heads and tokens (no GPU, nothing
launched), under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os

import pytest

from conftest import ROOT
from test_block_sanitizers_cpu import HIPCC, SAN_ENV, run

DRIVER = os.path.join(ROOT, "tests", "sanitize", "shape_driver.cpp")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(DRIVER)),
                    reason="needs the ROCm toolchain and the driver's source")
def test_every_shape_fits(tmp_path):
    csrc = os.path.join(ROOT, "activation_compression_pamm_amd", "csrc")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=all"]
    exe = str(tmp_path / "shapes")
    run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-x", "hip", DRIVER, "-o", exe])
    assert "shape driver ok" in run([exe], env=SAN_ENV).stdout
