"""AddressSanitizer + UndefinedBehaviorSanitizer on the host side of the block
operators' C ABI, on the CPU: sizes and strides at their extremes, every kind
of refusal, the workspace layouts and the clipping call's lists, with launchers
that check their arguments in place of the kernels' (no GPU, no device code)."""
import os

import pytest

from conftest import ROOT
from test_sanitizers_cpu import HIPCC, SAN_ENV, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs the ROCm toolchain")
def test_block_abi_host_side_under_asan_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "activation_compression_pamm_amd", "csrc")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    exe = str(tmp_path / "block_san")
    run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-x", "hip",
         os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp"), os.path.join(csrc, "pamm_block_api.hip"),
         "-o", exe])
    assert "block ABI sanitizer driver ok" in run([exe], env=SAN_ENV).stdout
