"""AddressSanitizer + UndefinedBehaviorSanitizer on the host side of the C ABI
of positions and of the cache in 8 bits, on the CPU: sizes and strides at their
extremes and the workspace layouts, with launchers that check their arguments
in place of the kernels' (no GPU, no device code)."""
import os

import pytest

from conftest import ROOT
from test_block_sanitizers_cpu import HIPCC, SAN_ENV, run

DRIVER = os.path.join(ROOT, "tests", "sanitize", "serving_driver.cpp")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(DRIVER)),
                    reason="needs the ROCm toolchain and the driver's source")
def test_serving_abi_host_side_under_asan_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "activation_compression_pamm_amd", "csrc")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    exe = str(tmp_path / "serving_san")
    run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-x", "hip", DRIVER,
         os.path.join(csrc, "pamm_rotary_api.hip"), os.path.join(csrc, "pamm_cache_api.hip"), "-o", exe])
    assert "serving ABI sanitizer driver ok" in run([exe], env=SAN_ENV).stdout
