"""The norm at the ends of its range: the largest batch, and values whose steps
leave fp32's range although the result does not."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launches_cover_every_batch_host(tmp_path):
    """The split of a batch into launches, to the last row of the largest batch
    (2^31 - 2 rows of 8 columns are accepted), tests/host/norm_rows_check.cpp."""
    exe = tmp_path / "norm_rows_check"
    src = os.path.join(ROOT, "tests", "host", "norm_rows_check.cpp")
    subprocess.run(["hipcc", "-O2", "-std=c++17", "-x", "hip", "--offload-arch=gfx950", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "moe_glue_amd", "csrc"), src, "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout + out.stderr
