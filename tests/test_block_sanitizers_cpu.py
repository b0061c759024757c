"""AddressSanitizer + UndefinedBehaviorSanitizer on the host side of the block
operators' C ABI, on the CPU: sizes and strides at their extremes, every kind
of refusal, the workspace layouts and the clipping call's lists, with launchers
that check their arguments in place of the kernels' (no GPU, no device code)."""
import os
import subprocess

import pytest

from conftest import ROOT

HIPCC = "/opt/rocm/bin/hipcc"
SAN_ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="-1")


def run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-3000:]}\n{r.stderr[-3000:]}"
    return r


DRIVER = os.path.join(ROOT, "tests", "sanitize", "block_driver.cpp")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(DRIVER)),
                    reason="needs the ROCm toolchain and the driver's source")
def test_block_abi_host_side_under_asan_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "activation_compression_pamm_amd", "csrc")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
           "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    exe = str(tmp_path / "block_san")
    run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
         "-packed-fp32-ops", *san, "-I", os.path.join(ROOT, "include"), "-I", csrc, "-x", "hip",
         DRIVER, os.path.join(csrc, "pamm_block_api.hip"),
         "-o", exe])
    assert "block ABI sanitizer driver ok" in run([exe], env=SAN_ENV).stdout
