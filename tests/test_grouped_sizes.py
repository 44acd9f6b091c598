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


def test_launches_host(tmp_path):
    """Every launch of the largest calls fits the runtime's limit on lanes, and a routing
    gradient's cover its tokens (tests/host/gradient_launches_check.cpp)."""
    exe = tmp_path / "gradient_launches_check"
    csrc = os.path.join(ROOT, "moe_glue_amd", "csrc")
    subprocess.run(["hipcc", "-O1", "-std=c++17", "-x", "hip", "--offload-arch=gfx950", "--cuda-host-only",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(ROOT, "tests", "host", "gradient_launches_check.cpp"),
                    *(os.path.join(csrc, f) for f in ("api.cpp", "grouped_linear.hip", "grouped_few.hip",
                                                      "grouped_grad.hip", "grads.hip")),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.endswith("ok\n"), f"status {out.returncode}: {out.stdout}{out.stderr}"


@pytest.mark.gpu
def test_routing_gradient_of_more_tokens_than_a_launch_holds():
    """2^26 + 3 tokens of 64 lanes each are more than 2^32.  With k = 2, weights 1/2 and dw =
    (a, b) the gradients are +- (a - b) / 4, and all are whole numbers of 32nds here."""
    import moe_glue_amd as mg

    dev, T = "cuda:0", 2 ** 26 + 3
    at = torch.arange(T, device=dev, dtype=torch.int32)
    ids = torch.stack((at % 2, 1 - at % 2), 1)
    dw = torch.stack((at % 61, at % 7), 1).float() / 8
    dlogits, none = mg.route_backward(ids, torch.full((T, 2), 0.5, device=dev), dw, 2)
    want = (dw[:, 0] - dw[:, 1]) / 4
    assert none is None and torch.equal(dlogits.gather(1, ids[:, :1].long())[:, 0], want)
    assert torch.equal(dlogits.gather(1, ids[:, 1:].long())[:, 0], -want)


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
