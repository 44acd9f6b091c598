"""The quantised norms' rows on their way to the experts: codes and scales through
the expand's row copy."""
import numpy as np
import pytest

import compare
import gpu_util as G
from moe_glue_amd import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,H,group", [("fp8", 512, 128), ("fp8", 2048, 128), ("fp8", 32, 8), ("mxfp8", 512, 32),
                                         ("mxfp8", 7168, 32)])
@pytest.mark.parametrize("T,pad_to", [(1, 1), (37, 1), (300, 16)])
def test_codes_and_scales_reach_expert_order(fmt, H, group, T, pad_to):
    import torch
    import moe_glue_amd as mg

    print(f"[norm to experts] {fmt} {T}x{H} group={group} pad_to={pad_to}", flush=True)
    dev = G.device()
    E, k = 12, 3
    rng = np.random.default_rng([T, H])
    x = inputs.f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    x[T // 2, H // 2] = 0x7FC0  # a NaN row: codes 0x7F, NaN scales
    w = inputs.f32_to_bf16_bits(rng.standard_normal(H).astype(np.float32))
    xd, wd = G.to_dev(x, dev), G.to_dev(w, dev)
    if fmt == "fp8":
        codes, scales, _ = mg.rmsnorm_fp8(xd, wd, group)
    else:
        codes, scales, _ = mg.rmsnorm_mxfp8(xd, wd)
    logits = G.to_dev(rng.standard_normal((T, E)).astype(np.float32), dev)
    r = mg.route_padded(logits, k, pad_to) if pad_to > 1 else mg.route(logits, k)
    rows = mg.padded_rows(T, E, k, pad_to) if pad_to > 1 else T * k
    dest = r["dest_of_src"].cpu().numpy()
    for name, t in (("codes", codes), ("scales", scales)):
        raw = t.view(torch.uint8)
        to = torch.full((rows, raw.shape[1] // 2), -1.0, dtype=torch.bfloat16, device=dev)
        mg.expand_rows(raw.view(torch.bfloat16), r["dest_of_src"], k, out=to)
        torch.cuda.synchronize()
        got = to.view(torch.uint8).cpu().numpy()
        compare.assert_equal(got[dest], np.repeat(raw.cpu().numpy(), k, 0), name)
        untouched = np.setdiff1d(np.arange(rows), dest)
        assert (got[untouched].reshape(-1, 2) == [0x80, 0xBF]).all(), f"{name}: padding rows"
