"""The grouped products at the ends of their sizes."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_host(tmp_path):
    """Arithmetic on sizes, trapping on signed overflow (tests/host/grouped_sizes_check.cpp).
    Host code alone: nothing of it runs a kernel, so what else the library has is left out."""
    exe = tmp_path / "grouped_sizes_check"
    csrc = os.path.join(ROOT, "moe_glue_amd", "csrc")
    trap = [f for flag in ("-fsanitize=signed-integer-overflow", "-fsanitize-trap=signed-integer-overflow")
            for f in ("-Xarch_host", flag)]
    subprocess.run(["hipcc", "-O1", "-std=c++17", "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only", *trap,
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(ROOT, "tests", "host", "grouped_sizes_check.cpp"),
                    *(os.path.join(csrc, f) for f in ("api.cpp", "grouped_linear.hip", "grouped_few.hip",
                                                      "grouped_grad.hip")),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.endswith("ok\n"), f"status {out.returncode} behind: {out.stdout}{out.stderr}"


@pytest.mark.gpu
def test_weight_gradient_of_the_most_rows():
    """2^31 - 8 rows of ones, the last 64: each piece's sums and the joined ones are whole
    numbers of at most 24 bits times a power of two, but for the last addition, which is
    off by half a step below 2^32 at most (128)."""
    import moe_glue_amd as mg

    R = 2 ** 31 - 8
    rows = torch.ones((R, 8), dtype=torch.bfloat16, device="cuda:0")     # 34 GB
    rows[-1] = 64.0
    dw, db = mg.grouped_linear_grad_w(rows, rows, dtype=torch.float32, bias=True)
    assert ((dw.double() - (R + 4095)).abs() <= 128).all(), dw[0, 0].item() - R
    assert ((db.double() - (R + 63)).abs() <= 128).all(), db[0].item() - R
