"""Every row kernel of the 8-bit product that is built can be launched (CPU only).

launch_rows (block_wise_bit_amd/csrc/dq4_int8_linear.hip) takes 16 weight rows at a
time (R = 1) only where a workgroup has no more than 16, and then there is no second row
block to keep a wave's codes in registers for (XF > 0)."""
import os
import re
import subprocess

from block_wise_bit_amd import build as dq4_build

SOURCE = next(s for s in dq4_build.SOURCES if os.path.basename(s) == "dq4_int8_linear.hip")
CUS = 256


def chosen(m, n, k):
    """(TF, R, XF) of an aligned call, or None where tiles take it."""
    if m > 64 or (m > 32 and k > 4096):
        return None
    tf = 1 if m <= 16 else 2 if m <= 32 else 4
    r = 2 if n > 16 * CUS else 1
    grid = min(-(-n // 16), CUS)
    steps = -(-(-(-k // 64)) // 8)
    if n <= grid * 16 * r:
        return tf, r, 0
    for xf, most in ((8, 4), (16, 2), (32, 1)):
        if steps <= xf and tf <= most:
            return tf, r, xf
    return tf, r, 0


def test_built_row_kernels_are_those_that_calls_take(tmp_path):
    out = tmp_path / "int8.s"
    subprocess.run([dq4_build.hipcc(), *dq4_build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I", dq4_build.INCLUDE, "-o",
                    str(out), SOURCE], check=True, cwd=tmp_path, stderr=subprocess.DEVNULL)
    built = {tuple(map(int, f)) for f in
             re.findall(r"16int8_rows_kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)EE", out.read_text())}
    sizes = (1, 16, 4096, 4097, 8192, 8193, 28672, 1 << 20)
    reached = {chosen(m, n, k) for m in (1, 16, 17, 32, 33, 64) for n in sizes
               for k in (16, 4096, 4112, 8192, 16384, 16400, 131056)} - {None}
    assert built == {(t, *c) for t in (1, 2) for c in reached}
