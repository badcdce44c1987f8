"""The host side of include/dq4_linear.h under AddressSanitizer and UBSan (host
code only: each -fsanitize= behind -Xarch_host).  No call of
tests/sanitize/linear_abi_driver.cpp reaches the GPU.  CPU only."""
import os
import subprocess

from block_wise_bit_amd import build as dq4_build

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.path.join(HERE, "sanitize")
# what the linear calls link against: the layout checks and the device queries
SOURCES = [s for s in dq4_build.SOURCES if os.path.basename(s) in ("dq4.hip", "dq4_linear_fused.hip")]


def test_linear_validation_and_plans_under_host_asan(tmp_path):
    exe = str(tmp_path / "linear_abi_driver")
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=undefined"]
    r = subprocess.run([dq4_build.hipcc(), *dq4_build.HIPCC_FLAGS, *host_san, "-g", "-I", dq4_build.INCLUDE, "-o", exe,
                        os.path.join(SAN, "linear_abi_driver.cpp"), *SOURCES], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:protect_shadow_gap=0"))
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "0 failures" in r.stdout
