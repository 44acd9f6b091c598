"""The norm held to the rounding of its own steps (plain64.NORM_STEPS_REL), and at
the ends of its range: the largest batch, and values whose steps leave fp32's range
although the result does not."""
import os
import subprocess

import numpy as np
import pytest

import compare
import gpu_util as G
import plain64 as P
from moe_glue_amd import inputs

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


@pytest.fixture(scope="module")
def dev():
    return G.device()


def bits(a):
    return inputs.f32_to_bf16_bits(np.asarray(a, np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 2048])
@pytest.mark.parametrize("steps", [3, 4, 5, 6])
def test_mxfp8_scale_of_a_maximum_just_below_2_128(dev, H, steps):
    """Half of a row is +-2, half +-1, so rms^2 = 5/2 + eps, and w = 1.6 * 2^127: eps
    puts the maximum `steps` fp32 steps below 2^128.  n is off by less than three, so
    it is finite and its scale that of a maximum below 2^128: 2^(127 - 8), the
    codes 448 (saturated) and 256 (255.99)."""
    import torch
    import moe_glue_amd as mg

    print(f"[norm top] H={H} steps={steps}", flush=True)
    rng = np.random.default_rng([H, steps])
    T = 3
    two = np.tile([2.0, 1.0], H // 2)
    sign = rng.choice([-1.0, 1.0], (T, H))
    w = bits(np.full(H, 1.6 * 2.0 ** 127))
    w64 = float((w[:1].astype(np.uint32) << 16).view(np.float32)[0])
    eps = (2 * (w64 * 2.0 ** -128) / (1 - steps * 2.0 ** -24)) ** 2 - 2.5
    assert 1e-3 < eps < 1  # so that its own rounding moves n by less than a sixteenth of a step
    codes, scales, _ = mg.rmsnorm_mxfp8(G.to_dev(bits(sign * two), dev), G.to_dev(w, dev), eps=eps)
    torch.cuda.synchronize()
    compare.assert_equal(scales.cpu().numpy(), np.full((T, H // 32), 246, np.uint8), "scales")
    want = np.where(two == 2, 0x7E, 0x78) | np.where(sign < 0, 0x80, 0)
    compare.assert_equal(codes.cpu().numpy(), want.astype(np.uint8), "codes")


@pytest.mark.gpu
def test_mxfp8_scale_where_x_times_w_passes_fp32(dev):
    """Rows of +-2^99 under w = 2^30 normalise to +-2^30 exactly, although the
    products of x and w pass fp32's range: scale 2^(30 - 8), code 256."""
    import torch
    import moe_glue_amd as mg

    rng = np.random.default_rng(0)
    T, H = 4, 1024
    sign = rng.choice([-1.0, 1.0], (T, H))
    codes, scales, _ = mg.rmsnorm_mxfp8(G.to_dev(bits(sign * 2.0 ** 99), dev), G.to_dev(bits(np.full(H, 2.0 ** 30)), dev))
    torch.cuda.synchronize()
    compare.assert_equal(scales.cpu().numpy(), np.full((T, H // 32), 127 + 22, np.uint8), "scales")
    compare.assert_equal(codes.cpu().numpy(), np.where(sign < 0, 0xF8, 0x78).astype(np.uint8), "codes")


@pytest.mark.gpu
@pytest.mark.parametrize("below", [True, False])
def test_mxfp8_scale_where_x_times_w_falls_below_fp32(dev, below):
    """One block of four holds +-15/4 * 2^-40, so rms = 15/8 * 2^-40 (eps aside); the
    others +-15/8 * 2^-105 under w = 2^-44: n = +-2^-109 times 1 / sqrt(1 + eps / rms^2),
    and x w, 15/8 * 2^-149, is no fp32.  With eps = 7e-8 * 2^-80 n lies 1e-8 of it below
    2^-109 and takes the scale 2^(-110 - 8), codes saturated; with the least eps,
    2^-48 of it away, 2^(-109 - 8), code 256."""
    import torch
    import moe_glue_amd as mg

    rng = np.random.default_rng(1)
    T, H = 3, 512
    sign = rng.choice([-1.0, 1.0], (T, H))
    big = np.arange(H) // 32 % 4 == 1
    x = sign * np.where(big, 3.75 * 2.0 ** -40, 1.875 * 2.0 ** -105)
    w = np.where(big, 1.0, 2.0 ** -44)
    eps = 7e-8 * 2.0 ** -80 if below else 1.2e-38
    codes, scales, _ = mg.rmsnorm_mxfp8(G.to_dev(bits(x), dev), G.to_dev(bits(w), dev), eps=eps)
    torch.cuda.synchronize()
    small = scales.cpu().numpy()[:, np.arange(H // 32) % 4 != 1]
    compare.assert_equal(small, np.full(small.shape, 127 - 117 - below, np.uint8), "scales")
    got = codes.cpu().numpy()[:, ~big]
    code = 0x7E if below else 0x78
    compare.assert_equal(got, np.where(sign[:, ~big] < 0, code | 0x80, code).astype(np.uint8), "codes")


def check_norm(dev, x, r, w, eps, fmt, group, what):
    """A call on bf16 bits, every output against the 64-bit form."""
    import torch
    import moe_glue_amd as mg

    T, H = x.shape
    s = (P.f64(x) + (0.0 if r is None else P.f64(r))).astype(np.float32).astype(np.float64)
    n = s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + np.float64(np.float32(eps))) * P.f64(w)
    xd, wd = G.to_dev(x, dev), G.to_dev(w, dev)
    rd = None if r is None else G.to_dev(r, dev)
    normed = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev)
    if fmt == "bf16":
        _, res = mg.rmsnorm(xd, wd, rd, eps, out=normed)
    elif fmt == "fp8":
        codes, scales, res = mg.rmsnorm_fp8(xd, wd, group, rd, eps, normed=normed)
    else:
        codes, scales, res = mg.rmsnorm_mxfp8(xd, wd, rd, eps, normed=normed)
    torch.cuda.synchronize()
    if r is not None:
        compare.assert_equal(G.to_host(res), bits(s.astype(np.float32)), f"{what}: residual_out")
    P.assert_within(P.f64(G.to_host(normed)), n, P.norm_steps_bound(n), f"{what}: out")
    if fmt == "bf16":
        return
    b = n.reshape(T, -1, group)
    amax = np.abs(b).max(-1)
    q = P.e4m3_values(codes.cpu().numpy()).reshape(b.shape)
    if fmt == "fp8":
        sc = scales.cpu().numpy().astype(np.float64)
        P.assert_within(sc, amax / 448, (P.NORM_STEPS_REL + P.FP32) * amax / 448 + P.FP32_TINY, f"{what}: scales")
    else:
        compare.assert_equal(scales.cpu().numpy().astype(int), P.mx_exponent(amax) + 127, f"{what}: scales")
        sc = 2.0 ** P.mx_exponent(amax)
        b = np.clip(b, -448 * sc[..., None], 448 * sc[..., None])
    P.assert_within(q * sc[..., None], b, P.quantised_steps_bound(b, sc[..., None]), f"{what}: codes")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", [("bf16", 0), ("fp8", 8), ("fp8", 64), ("mxfp8", 32)])
@pytest.mark.parametrize("H", [256, 2112, 8256])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_whose_quotient_falls_below_fp32(dev, fmt, group, H, residual):
    """Small values beside large ones under large weights: s / rms is below fp32's
    normals, or its whole range, n is not."""
    print(f"[norm low] {fmt} group={group} H={H} residual={residual}", flush=True)
    rng = np.random.default_rng([H, group, residual])
    big = np.arange(H) // 32 % 4 == 1
    w = np.where(big, 1.0, np.where(np.arange(H) % 2 == 0, 2.0 ** 100, 2.0 ** 127)) * rng.uniform(1, 1.9, H)
    #       rms about 2^40    2^100         subnormal x     about 2^-126   neighbours large and small
    rows = [(41.0, -100.0), (101.0, -120.0), (20.0, -130.0), (41.0, -86.0), (41.0, -100.0), (41.0, -100.0)]
    x = np.stack([np.where(big, 2.0 ** hi, 2.0 ** lo) for hi, lo in rows])
    x[4, 5::8] = 2.0 ** 41   # (their own weights large: n up to 2^128 / 4)
    w[5::8] = np.minimum(w[5::8], 2.0 ** 100)
    x[5, ::3] = 0
    x = x * rng.uniform(1, 1.9, x.shape) * rng.choice([-1, 1], x.shape)
    r = np.where(rng.random(x.shape) < 0.5, x * rng.uniform(-1, 1, x.shape), 0) if residual else None
    check_norm(dev, bits(x), None if r is None else bits(r), bits(w), 1e-6, fmt, group, f"{fmt} {H}")


NORM_SIZES = [("bf16", 0, 1, 8), ("bf16", 0, 7, 520), ("bf16", 0, 40, 2048), ("bf16", 0, 9, 8200), ("bf16", 0, 2, 65536),
              ("fp8", 8, 3, 24), ("fp8", 128, 40, 2048), ("fp8", 512, 9, 7168), ("fp8", 64, 3, 16448),
              ("mxfp8", 32, 3, 96), ("mxfp8", 32, 40, 2048), ("mxfp8", 32, 9, 7168), ("mxfp8", 32, 2, 65536)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group,T,H", NORM_SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_is_right_to_its_roundings(dev, fmt, group, T, H, residual):
    """Rows from 2^-60 to 2^60: the scales, which are not rounded to 8 bits, see an
    error of a few fp32 steps in the row's sum."""
    print(f"[norm steps] {fmt} group={group} {T}x{H} residual={residual}", flush=True)
    rng = np.random.default_rng([T, H, group, residual])
    row = 2.0 ** np.linspace(-60, 60, T)[:, None]
    x = bits(row * rng.standard_normal((T, H)))
    r = bits(4 * row * rng.standard_normal((T, H))) if residual else None
    check_norm(dev, x, r, bits(rng.standard_normal(H)), 1e-30, fmt, group, f"{fmt} {T}x{H}")
