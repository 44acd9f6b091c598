"""The README's Python examples run as printed."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def examples():
    text = open(os.path.join(ROOT, "README.md")).read()
    return re.findall(r"^```python\n(.*?)^```", text, flags=re.S | re.M)


def test_examples_compile():
    blocks = examples()
    assert len(blocks) >= 2
    for i, code in enumerate(blocks):
        compile(code, f"README.md example {i}", "exec")


@pytest.mark.gpu
def test_examples_run_in_order():
    import torch

    space = {}
    for i, code in enumerate(examples()):
        print(f"[readme] example {i}", flush=True)
        exec(compile(code, f"README.md example {i}", "exec"), space)
        torch.cuda.synchronize()
    T, H = 32, space["H"]
    assert space["out"].shape == (4096, H) and space["normed"].shape == space["res"].shape == (T, H)
    for key in ("r", "r4"):
        out = space[key]["out"]
        assert out.shape == (T, H) and bool(out.isfinite().all()) and bool((out != 0).any())
