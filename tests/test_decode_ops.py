"""The norm, the MXFP4 linear and the few-token layer on an MI355X against their
64-bit forms (tests/plain64.py)."""
import sys

import numpy as np
import pytest

import compare
import gpu_util as G
import plain64 as P
from moe_glue_amd import inputs

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def dev():
    return G.device()


def bf16(rng, shape, std=1.0):
    return inputs.f32_to_bf16_bits((std * rng.standard_normal(shape)).astype(np.float32))


def host(t):
    return P.f64(G.to_host(t)) if str(t.dtype) == "torch.bfloat16" else t.cpu().numpy()


# ------------------------------------------------------------------- norm
def norm_inputs(T, H, seed, special=False):
    rng = np.random.default_rng([7, T, H, seed])
    x, r = bf16(rng, (T, H)), bf16(rng, (T, H), 4.0)
    w = bf16(rng, (H,), 0.2)
    if special:  # rows at the edges of fp32, one row each
        big = np.array([1e30, 3e38, 1e-30, 1e-38, 1e-41], np.float32)
        for i, v in enumerate(big):
            x[i] = inputs.f32_to_bf16_bits(v * rng.choice([-1, 1], H).astype(np.float32))
            r[i] = 0
        x[5], r[5] = 0, 0
        x[6, 3] = 0x7F80  # +inf
        x[7, 5] = 0x7FC0  # NaN
        x[8], r[8] = x[9], x[9] ^ 0x8000  # x = -r: a sum of zeros
    return x, r, w


def check_norm(dev, T, H, fmt, group, residual, normed, inplace=False, special=False, seed=0):
    import torch
    import moe_glue_amd as mg

    x, r, w = norm_inputs(T, H, seed, special)
    if not residual:
        r = None
    s, n = P.rmsnorm(x, r, w, EPS)
    xd, wd = G.to_dev(x, dev), G.to_dev(w, dev)
    rd = G.to_dev(r, dev) if residual else None
    ro = rd if inplace else None
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev) if normed or fmt == "bf16" else None
    if fmt == "bf16":
        out, res = mg.rmsnorm(xd, wd, rd, EPS, out=out, residual_out=ro)
    elif fmt == "fp8":
        codes, scales, res = mg.rmsnorm_fp8(xd, wd, group, rd, EPS, residual_out=ro, normed=out)
    else:
        codes, scales, res = mg.rmsnorm_mxfp8(xd, wd, rd, EPS, residual_out=ro, normed=out)
    torch.cuda.synchronize()
    what = f"norm {fmt} {T}x{H}"
    if residual:
        with np.errstate(over="ignore", invalid="ignore"):
            want = inputs.f32_to_bf16_bits((P.f64(x) + P.f64(r)).astype(np.float32))
        fine = np.isfinite(s).all(-1)
        compare.assert_equal(G.to_host(res)[fine], want[fine], f"{what}: residual_out")
        assert res is rd if inplace else True
    else:
        assert res is None
    if out is not None:
        P.assert_within(host(out), n, P.rmsnorm_bound(n), f"{what}: out")
    if fmt == "bf16":
        return
    b = n.reshape(T, -1, group)
    fine = np.isfinite(b).all(-1)
    amax = np.abs(b).max(-1)
    q = P.e4m3_values(codes.cpu().numpy()).reshape(b.shape)
    assert np.isnan(q[~fine]).all()
    if fmt == "fp8":
        sc = scales.cpu().numpy().astype(np.float64)
        assert np.isnan(sc[~fine]).all()
        P.assert_within(sc[fine], (amax / 448)[fine], (2 * P.NORM_REL * amax / 448 + 2.0 ** -149)[fine], f"{what}: scales")
    else:
        by = scales.cpu().numpy().astype(np.float64)
        assert (by[~fine] == 255).all()
        sc = 2.0 ** (by - 127)
        # floor(log2 amax) - 8, of an amax that the kernel has to NORM_REL
        with np.errstate(divide="ignore"):
            lo = np.maximum(np.floor(np.log2(amax * (1 - 2 * P.NORM_REL))) - 8, -127)
            hi = np.maximum(np.floor(np.log2(amax * (1 + 2 * P.NORM_REL))) - 8, -127)
        ok = (by - 127 >= lo) & (by - 127 <= hi)
        assert ok[fine].all(), f"{what}: scale bytes"
        # magnitudes in (448, 512) of a block's scale saturate
        sat = 448.0 * sc[..., None]
        b = np.clip(b, -sat, sat)
    s3 = sc[..., None]
    with np.errstate(invalid="ignore"):
        P.assert_within((q * s3)[fine], b[fine], P.quantised_bound(b, s3)[fine], f"{what}: codes")


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 16), (7, 520), (5, 2048), (2, 2056), (3, 4096), (2, 4104), (3, 7168),
                                 (2, 8192), (1, 8200), (1, 16384), (1, 16392), (2, 65536), (1031, 256)])
def test_rmsnorm(dev, T, H, residual):
    _log(f"[norm] {T}x{H} residual={residual}")
    check_norm(dev, T, H, "bf16", 0, residual, True)


@pytest.mark.parametrize("T,H,group", [(1, 8, 8), (3, 16, 16), (7, 520, 8), (5, 2048, 128), (3, 4096, 512),
                                       (2, 4160, 64), (3, 7168, 256), (2, 16896, 512), (1, 65536, 32), (513, 256, 32)])
def test_rmsnorm_fp8(dev, T, H, group):
    _log(f"[norm fp8] {T}x{H} group={group}")
    check_norm(dev, T, H, "fp8", group, True, True)
    check_norm(dev, T, H, "fp8", group, False, False, seed=1)


@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (5, 2048), (2, 2080), (3, 7168), (2, 8224), (1, 65536), (513, 256)])
def test_rmsnorm_mxfp8(dev, T, H):
    _log(f"[norm mxfp8] {T}x{H}")
    check_norm(dev, T, H, "mxfp8", 32, True, True)
    check_norm(dev, T, H, "mxfp8", 32, False, False, seed=1)


@pytest.mark.parametrize("fmt,group", [("bf16", 0), ("fp8", 128), ("mxfp8", 32)])
@pytest.mark.parametrize("H", [512, 2048, 12800])
def test_rmsnorm_special_rows_and_in_place(dev, fmt, group, H):
    """Rows of squares beyond and below fp32, zeros, an infinity, a NaN; the
    residual updated in its own buffer."""
    _log(f"[norm special] {fmt} H={H}")
    check_norm(dev, 10, H, fmt, group, True, True, inplace=True, special=True)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8"])
def test_rmsnorm_codes_bit_exact_where_n_is_a_bf16(dev, oracle_lib, fmt):
    """Rows of +-2^a with eps far below their squares normalise to +-1 exactly,
    so n = +-w is a bf16 row: codes and scales are the quantising expand's."""
    import torch
    import moe_glue_amd as mg

    T, H, group = 6, 1024, 64
    rng = np.random.default_rng(5)
    sign = rng.choice([-1.0, 1.0], (T, H))
    x = inputs.f32_to_bf16_bits((sign * 2.0 ** np.arange(-2, T - 2)[:, None]).astype(np.float32))
    w = bf16(rng, (H,), 3.0)
    w[:64] = 0  # an all-zero group
    w[64:128] = 0x3F80  # a group on its maximum
    n = inputs.f32_to_bf16_bits((sign * P.f64(w)).astype(np.float32))
    ident = np.arange(T, dtype=np.int32)
    xd, wd = G.to_dev(x, dev), G.to_dev(w, dev)
    if fmt == "fp8":
        codes, scales, _ = mg.rmsnorm_fp8(xd, wd, group, eps=1e-30)
        qr, sr = oracle_lib.expand_rows_fp8(n, ident, 1, group)
    else:
        codes, scales, _ = mg.rmsnorm_mxfp8(xd, wd, eps=1e-30)
        qr, sr = oracle_lib.expand_rows_mxfp8(n, ident, 1)
    torch.cuda.synchronize()
    compare.assert_equal(codes.cpu().numpy(), qr, "codes")
    compare.assert_equal(scales.cpu().numpy(), sr, "scales")


@pytest.mark.parametrize("H", [32, 2048, 7168])
def test_rmsnorm_mxfp8_scale_of_a_maximum_just_below_a_power_of_two(dev, H):
    """Rows of +-15/8 normalise to +-1 / sqrt(1 + eps / R), R = 225/64: with eps =
    7e-8 that is 1 - 1e-8, which fp32 would round to 1.  Its scale is still that
    of a maximum below 1 (2^-9, codes saturated); without eps to speak of n is 1
    (2^-8, code 256)."""
    import torch
    import moe_glue_amd as mg

    rng = np.random.default_rng(H)
    T = 4
    sign = rng.choice([-1.0, 1.0], (T, H))
    x = G.to_dev(inputs.f32_to_bf16_bits((1.875 * sign).astype(np.float32)), dev)
    shift = rng.integers(-3, 4, H // 32)  # blocks of w = 2^j
    w = G.to_dev(inputs.f32_to_bf16_bits(np.repeat(2.0 ** shift, 32).astype(np.float32)), dev)
    for eps, exponent, code in ((7e-8, -9, 0x7E), (2e-38, -8, 0x78)):
        codes, scales, _ = mg.rmsnorm_mxfp8(x, w, eps=eps)
        torch.cuda.synchronize()
        compare.assert_equal(scales.cpu().numpy().astype(int), np.tile(127 + exponent + shift, (T, 1)), f"eps {eps}")
        compare.assert_equal(codes.cpu().numpy(), np.where(sign < 0, code | 0x80, code).astype(np.uint8), f"eps {eps}")


def test_rmsnorm_row_does_not_depend_on_its_batch(dev):
    import torch
    import moe_glue_amd as mg

    for H in (2048, 7168):
        x, r, w = norm_inputs(1500, H, 3)
        xd, rd, wd = (G.to_dev(v, dev) for v in (x, r, w))
        out, res = mg.rmsnorm(xd, wd, rd)
        for n in (1, 40, 700):
            o, s = mg.rmsnorm(xd[:n].contiguous(), wd, rd[:n].contiguous())
            assert torch.equal(o.view(torch.int16), out[:n].view(torch.int16))
            assert torch.equal(s.view(torch.int16), res[:n].view(torch.int16))


def test_norm_and_linear_and_layer_take_empty_batches(dev):
    import torch
    import moe_glue_amd as mg

    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    u8 = torch.uint8
    assert mg.rmsnorm(e(0, 64), e(64))[0].shape == (0, 64)
    assert mg.rmsnorm_fp8(e(0, 64), e(64), 32, e(0, 64))[0].shape == (0, 64)
    assert mg.rmsnorm_mxfp8(e(0, 64), e(64))[1].shape == (0, 2)
    assert mg.linear_mxfp4(e(0, 64), e(5, 32, dt=u8), e(5, 2, dt=u8)).shape == (0, 5)
    r = mg.decode_layer(e(0, 4, dt=torch.float32), 2, e(0, 64), e(4, 64, 64), e(4, 64, 32))
    assert r["out"].shape == (0, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
@pytest.mark.parametrize("T,H", [((1 << 22) + 5, 32), (70001, 32768)])
def test_rmsnorm_many_rows(dev, fmt, T, H):
    """More rows than one launch takes, and tensors past 2^32 bytes: the last rows
    are what they are alone."""
    import torch
    import moe_glue_amd as mg

    _log(f"[norm many] {fmt} {T}x{H}")
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(dev).manual_seed(3))
    w = torch.ones(H, dtype=torch.bfloat16, device=dev) * 1.5
    call = {"bf16": lambda v: mg.rmsnorm(v, w)[:1], "fp8": lambda v: mg.rmsnorm_fp8(v, w, 32)[:2],
            "mxfp8": lambda v: mg.rmsnorm_mxfp8(v, w)[:2]}[fmt]
    whole = call(x)
    for lo, hi in ((0, 3), ((1 << 21) - 1, (1 << 21) + 2), (T - 7, T)):
        if hi <= T:
            for a, b in zip(whole, call(x[lo:hi].contiguous())):
                assert torch.equal(a[lo:hi].view(torch.uint8), b.view(torch.uint8)), (lo, hi)


# ------------------------------------------------------------------ MXFP4
def mxfp4(rng, shape, lo=118, hi=122):
    *lead, K = shape
    return (rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*lead, K // 32), dtype=np.uint8))


def test_linear_mxfp4_every_code_and_scale(dev):
    """x picks single weights, so y is the weight itself: every code under every
    scale byte up to 252 (subnormal bf16 at the low end) exactly, NaN for 255."""
    import torch
    import moe_glue_amd as mg

    N, K = 256, 32
    codes = np.tile(np.array([(2 * i + 1) << 4 | 2 * i for i in range(8)] * 2, np.uint8), (N, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    x = np.zeros((K, K), np.uint16)
    x[np.arange(K), np.arange(K)] = 0x3F80
    y = host(mg.linear_mxfp4(*(G.to_dev(v, dev) for v in (x, codes, scales))))
    want = P.mxfp4_values(codes, scales).T
    assert np.array_equal(y[:, :253], want[:, :253])
    assert np.isnan(y[:, 255]).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,K,N", [(1, 32, 1), (1, 64, 17), (2, 96, 5), (5, 128, 33), (16, 160, 16), (17, 256, 15),
                                   (31, 2048, 70), (33, 1056, 31), (48, 992, 64), (64, 7168, 50), (64, 4096, 130),
                                   (1, 7168, 4096), (7, 16384, 19), (20, 96, 4097), (40, 1312, 5000), (9, 288, 4104),
                                   (5, 544, 8196), (33, 160, 8193), (64, 2016, 1030), (17, 256, 1028), (12, 32, 6001),
                                   (64, 4128, 8200), (17, 96, 2050), (33, 1056, 4095), (64, 160, 3001),
                                   (13, 2336, 8195), (6, 2080, 8300)])
def test_linear_mxfp4(dev, T, K, N):
    import torch
    import moe_glue_amd as mg

    _log(f"[linear] T={T} K={K} N={N}")
    rng = np.random.default_rng([3, T, K, N])
    x = bf16(rng, (T, K))
    w, s = mxfp4(rng, (N, K), 100, 150)
    pad = torch.full((T * N + 64,), 0x7B7B, dtype=torch.int16, device=dev)
    out = pad[:T * N].view(torch.bfloat16).view(T, N)
    mg.linear_mxfp4(G.to_dev(x, dev), G.to_dev(w, dev), G.to_dev(s, dev), out=out)
    torch.cuda.synchronize()
    y, bound = P.linear(x, P.mxfp4_values(w, s))
    P.assert_within(host(out), y, bound, f"linear {T}x{K}x{N}")
    assert (pad[T * N:] == 0x7B7B).all(), "wrote past y"


# ------------------------------------------------------------------ layer
def layer_inputs(T, E, k, H, I, fmt, seed=0, kind="normal"):
    rng = np.random.default_rng([11, T, E, k, H, I, seed])
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "same":      # every token picks the same experts
        logits = np.tile(logits[:1], (T, 1))
    elif kind == "ties":
        logits = inputs.quantized_logits(T, E, seed)
    bias = (0.5 * rng.standard_normal(E)).astype(np.float32) if kind == "bias" else None
    x = bf16(rng, (T, H))
    if fmt == "bf16":
        wgu, wd = bf16(rng, (E, 2 * I, H), H ** -0.5), bf16(rng, (E, H, I), I ** -0.5)
        return logits, bias, x, (wgu, wd), (P.f64(wgu), P.f64(wd))
    wgu, sgu = mxfp4(rng, (E, 2 * I, H))
    wd, sd = mxfp4(rng, (E, H, I))
    return logits, bias, x, (wgu, sgu, wd, sd), (P.mxfp4_values(wgu, sgu), P.mxfp4_values(wd, sd))


def run_layer(mg, k, logits, bias, x, w, out=None):
    call = mg.decode_layer if len(w) == 2 else mg.decode_layer_mxfp4
    return call(logits, k, x, *w, bias=bias, out=out)


def guarded_outputs(mg, T, E, k, H, I, dev, fill):
    """Outputs and a workspace of exactly the documented size, garbage-filled,
    each with guard bytes behind it."""
    import torch

    def buf(shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 256,), fill, dtype=torch.uint8, device=dev)
        return raw, raw[:n].view(dtype).view(shape)

    raws, out = {}, {}
    for key, shape, dtype in (("topk_ids", (T, k), torch.int32), ("topk_weights", (T, k), torch.float32),
                              ("out", (T, H), torch.bfloat16),
                              ("workspace", (mg.decode_layer_workspace_bytes(T, E, k, I),), torch.uint8)):
        raws[key], out[key] = buf(shape, dtype)
    return raws, out


LAYER_SHAPES = [(1, 1, 1, 8, 8), (3, 4, 2, 16, 8), (16, 8, 2, 256, 128), (1, 128, 8, 2048, 768), (5, 17, 5, 520, 72),
                (64, 4, 4, 128, 40), (64, 8, 1, 64, 64), (33, 12, 12, 96, 48), (64, 40, 16, 72, 24),
                (64, 512, 16, 64, 32), (13, 64, 6, 1408, 264), (2, 3, 2, 4104, 24), (32, 32, 8, 200, 520)]
LAYER4_SHAPES = [(1, 1, 1, 32, 32), (3, 4, 2, 64, 32), (16, 8, 2, 256, 128), (1, 32, 8, 2048, 768),
                 (5, 17, 5, 544, 96), (64, 4, 4, 128, 160), (64, 8, 1, 64, 64), (33, 12, 12, 96, 32),
                 (64, 40, 16, 96, 32), (64, 512, 16, 64, 32), (13, 64, 6, 1056, 288), (32, 32, 8, 224, 544)]


@pytest.mark.parametrize("fmt,shape", [("bf16", s) for s in LAYER_SHAPES] + [("mxfp4", s) for s in LAYER4_SHAPES],
                         ids=str)
@pytest.mark.parametrize("kind", ["normal", "same", "ties", "bias"])
def test_decode_layer(dev, fmt, shape, kind):
    import torch
    import moe_glue_amd as mg

    T, E, k, H, I = shape
    _log(f"[layer] {fmt} T={T} E={E} k={k} H={H} I={I} {kind}")
    logits, bias, x, w, w64 = layer_inputs(T, E, k, H, I, fmt, kind=kind)
    ids, weights = P.route(logits if bias is None else logits + bias, k)
    raws, out = guarded_outputs(mg, T, E, k, H, I, dev, 0xC5)
    b = None if bias is None else G.to_dev(bias, dev)
    args = (G.to_dev(logits, dev), b, G.to_dev(x, dev), [G.to_dev(v, dev) for v in w])
    run_layer(mg, k, *args, out=out)
    torch.cuda.synchronize()
    first = {key: raw.cpu().numpy().copy() for key, raw in raws.items()}
    compare.assert_equal(out["topk_ids"].cpu().numpy(), ids, "topk_ids")
    compare.assert_weights_close(out["topk_weights"].cpu().numpy(), weights)
    want, bound = P.layer(x, ids, weights, *w64)
    P.assert_within(host(out["out"]), want, bound, f"layer {fmt} {shape}")
    for key, raw in raws.items():
        assert (raw[-256:] == 0xC5).all(), f"wrote past {key}"
    run_layer(mg, k, *args, out=out)  # over its own left-overs: the same bits
    torch.cuda.synchronize()
    for key in ("topk_ids", "topk_weights", "out"):
        assert np.array_equal(first[key], raws[key].cpu().numpy()), f"{key} changed on the second call"


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_decode_layer_of_experts_past_32_bits(dev, fmt):
    """Weights of more than 2^32 bytes (and 2^32 values): the last experts give
    what they give in a tensor of their own."""
    import torch
    import moe_glue_amd as mg

    E, few, k, H, I = 160, 4, 2, 8192, 2048
    _log(f"[layer big] {fmt} E={E} H={H} I={I}")
    rng = np.random.default_rng(9)
    T = 5
    x = G.to_dev(bf16(rng, (T, H)), dev)
    small_logits = rng.standard_normal((T, few)).astype(np.float32)
    logits = np.full((T, E), -50.0, np.float32)
    logits[:, E - few:] = small_logits
    if fmt == "bf16":
        last = [G.to_dev(bf16(rng, s, 0.02), dev) for s in ((few, 2 * I, H), (few, H, I))]
    else:
        last = [G.to_dev(v, dev) for s in ((few, 2 * I, H), (few, H, I)) for v in mxfp4(rng, s)]
    big = []
    for v in last:
        t = torch.zeros((E, *v.shape[1:]), dtype=v.dtype, device=dev)
        t[E - few:] = v
        big.append(t)
    a = run_layer(mg, k, G.to_dev(logits, dev), None, x, big)
    b = run_layer(mg, k, G.to_dev(small_logits, dev), None, x, last)
    torch.cuda.synchronize()
    assert torch.equal(a["topk_ids"], b["topk_ids"] + (E - few))
    assert torch.equal(a["out"].view(torch.int16), b["out"].view(torch.int16))


@pytest.mark.parametrize("T,K,N", [(3, 96, 33), (8, 288, 70), (20, 96, 4100), (33, 544, 8197)])
def test_linear_mxfp4_nan_stays_in_its_token_and_row(dev, T, K, N):
    import torch
    import moe_glue_amd as mg

    _log(f"[linear nan] T={T} K={K} N={N}")
    rng = np.random.default_rng(T)
    x = bf16(rng, (T, K))
    w, sc = mxfp4(rng, (N, K))
    clean = G.to_host(mg.linear_mxfp4(*(G.to_dev(v, dev) for v in (x, w, sc))))
    x[1, K - 1], x[2, 0] = 0x7FC0, 0x7F80  # NaN, infinity
    sc[N - 1, K // 32 - 1] = 255
    sc[5, 0] = 255
    got = G.to_host(mg.linear_mxfp4(*(G.to_dev(v, dev) for v in (x, w, sc))))
    rows = [n for n in range(N) if n not in (5, N - 1)]
    tokens = [t for t in range(T) if t not in (1, 2)]
    assert np.array_equal(got[tokens][:, rows], clean[tokens][:, rows])
    isnan = (got & 0x7FFF) > 0x7F80
    assert isnan[:, [5, N - 1]].all() and isnan[1].all()
    assert ((got[2] & 0x7FFF) >= 0x7F80).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,H,I", [(1, 96, 32), (9, 96, 160), (40, 288, 96), (64, 4128, 64)])
def test_decode_layer_nan_stays_in_its_token_and_expert(dev, fmt, T, H, I):
    import torch
    import moe_glue_amd as mg

    _log(f"[layer nan] {fmt} T={T} H={H} I={I}")
    E, k = 6, 2
    rng = np.random.default_rng(T + H)
    x = bf16(rng, (T, H))
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if fmt == "bf16":
        w = [bf16(rng, (E, 2 * I, H), 0.1), bf16(rng, (E, H, I), 0.1)]
    else:
        w = [v for s in ((E, 2 * I, H), (E, H, I)) for v in mxfp4(rng, s)]
    on = lambda v: G.to_dev(v, dev)
    ld, dev_w = on(logits), [on(v) for v in w]
    clean = run_layer(mg, k, ld, None, on(x), dev_w)
    ids, out = G.to_host(clean["topk_ids"]), G.to_host(clean["out"])
    bad = ids[0, 0]
    t = T - 1
    poisoned = x.copy()
    poisoned[t, H - 1] = 0x7FC0
    got = G.to_host(run_layer(mg, k, ld, None, on(poisoned), dev_w)["out"])
    assert np.array_equal(got[:t], out[:t]) and ((got[t] & 0x7FFF) > 0x7F80).all()

    # one row of the expert's up weights: all outputs of its tokens; one row of its
    # down weights: that output of them
    routed = (ids == bad).any(axis=1)
    for which, row, columns in ((0, 2 * I - 1, slice(None)), (1, H - 2, slice(H - 2, H - 1))):
        v = [a.copy() for a in w]
        if fmt == "bf16":
            v[which][bad, row, -1] = 0x7FC0
        else:
            v[2 * which + 1][bad, row, -1] = 255
        got = G.to_host(run_layer(mg, k, ld, None, on(x), [on(a) for a in v])["out"])
        want = np.zeros(got.shape, bool)
        want[routed, columns] = True
        assert np.array_equal((got & 0x7FFF) > 0x7F80, want)
        assert np.array_equal(got[~want], out[~want])
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 9, 64])
def test_layer_matches_the_separate_calls(dev, T):
    """The layer against the path's separate calls with library products between
    them: the two round at different places, so each is held to its own bound."""
    import torch
    import moe_glue_amd as mg

    E, k, H, I = 16, 4, 512, 256
    logits, _, x, w, w64 = layer_inputs(T, E, k, H, I, "bf16")
    ld, xd, wgu, wd = (G.to_dev(v, dev) for v in (logits, x, *w))
    got = mg.decode_layer(ld, k, xd, wgu, wd)
    r = mg.route_expand(ld, k, xd)
    off = r["expert_offsets"].cpu().numpy()
    h = torch.empty((T * k, 2 * I), dtype=torch.bfloat16, device=dev)
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
    for e in range(E):
        h[off[e]:off[e + 1]] = (r["x_expanded"][off[e]:off[e + 1]].float() @ wgu[e].float().T).bfloat16()
    act = mg.swiglu(h)
    for e in range(E):
        y[off[e]:off[e + 1]] = (act[off[e]:off[e + 1]].float() @ wd[e].float().T).bfloat16()
    ref = mg.combine(y, r["topk_weights"], r["dest_of_src"])
    torch.cuda.synchronize()
    assert torch.equal(got["topk_ids"], r["topk_ids"]) and torch.equal(got["topk_weights"], r["topk_weights"])
    ids, weights = P.route(logits, k)
    want, bound = P.layer(x, ids, weights, *w64)
    P.assert_within(host(got["out"]), want, bound, "layer")
    # h's and y's own roundings on top
    sum_w = np.abs(want) * 0 + 1
    assert np.sqrt(np.mean((host(ref) - host(got["out"])) ** 2)) <= 4 * P.BF16 * np.sqrt(np.mean(want ** 2)) * sum_w.max()


def decode_block(mg, torch, st, bufs):
    """One decode step round a layer: residual and norm, router, experts and a
    shared expert, residual and norm for the next product."""
    normed, res = mg.rmsnorm(st["x"], st["w1"], st["r"], out=bufs["normed"], residual_out=bufs["res"])
    torch.mm(normed.float(), st["wr"], out=bufs["logits"])
    lay = mg.decode_layer_mxfp4(bufs["logits"], st["k"], normed, *st["experts"], out=bufs["layer"])
    h = mg.linear_mxfp4(normed, *st["shared_gu"], out=bufs["h"])
    act = mg.swiglu(h, out=bufs["act"])
    sh = mg.linear_mxfp4(act, *st["shared_d"], out=bufs["sh"])
    torch.add(lay["out"], sh, out=bufs["sum"])
    return mg.rmsnorm_mxfp8(bufs["sum"], st["w2"], res, out=bufs["codes"], scales=bufs["scales"], residual_out=res,
                            normed=bufs["last"])


def block_state(mg, torch, T, dev, seed=0):
    E, k, H, I = 16, 4, 256, 96
    rng = np.random.default_rng([23, seed])
    d = lambda a: G.to_dev(a, dev)  # noqa: E731
    st = {"k": k, "x": d(bf16(rng, (T, H))), "r": d(bf16(rng, (T, H))), "w1": d(bf16(rng, (H,))),
          "w2": d(bf16(rng, (H,))), "wr": d(rng.standard_normal((H, E)).astype(np.float32) * np.float32(H ** -0.5)),
          "experts": [d(v) for s in ((E, 2 * I, H), (E, H, I)) for v in mxfp4(rng, s)],
          "shared_gu": [d(v) for v in mxfp4(rng, (2 * I, H))], "shared_d": [d(v) for v in mxfp4(rng, (H, I))]}
    b = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    bufs = {"normed": b(T, H), "res": b(T, H), "logits": b(T, E, dt=torch.float32),
            "layer": mg.alloc_decode_outputs(T, E, k, H, I, dev), "h": b(T, 2 * I), "act": b(T, I), "sh": b(T, H),
            "sum": b(T, H), "codes": b(T, H, dt=torch.uint8), "scales": b(T, H // 32, dt=torch.uint8),
            "last": b(T, H)}
    return st, bufs, (E, k, H, I)


@pytest.mark.parametrize("T", [1, 6, 64])
def test_decode_block_step_by_step(dev, T):
    """The operators as a decode step chains them, each against its 64-bit form
    on the inputs that it had."""
    import torch
    import moe_glue_amd as mg

    st, bufs, (E, k, H, I) = block_state(mg, torch, T, dev)
    decode_block(mg, torch, st, bufs)
    torch.cuda.synchronize()
    hb = {key: G.to_host(v) for key, v in bufs.items() if key != "layer"}
    hs = {key: G.to_host(v) for key, v in st.items() if hasattr(v, "dtype")}
    lay = {key: G.to_host(v) for key, v in bufs["layer"].items()}
    s, n = P.rmsnorm(hs["x"], hs["r"], hs["w1"], 1e-6)
    P.assert_within(P.f64(hb["normed"]), n, P.rmsnorm_bound(n), "first norm")
    ids, weights = P.route(hb["logits"], k)
    compare.assert_equal(lay["topk_ids"], ids, "ids")
    ex = [G.to_host(v) for v in st["experts"]]
    want, bound = P.layer(hb["normed"], ids, weights, P.mxfp4_values(*ex[:2]), P.mxfp4_values(*ex[2:]))
    P.assert_within(P.f64(lay["out"]), want, bound, "layer")
    for name, x, w, got in (("shared gate-up", "normed", "shared_gu", "h"), ("shared down", "act", "shared_d", "sh")):
        y, bd = P.linear(hb[x], P.mxfp4_values(*(G.to_host(v) for v in st[w])))
        P.assert_within(P.f64(hb[got]), y, bd, name)
    sbits = inputs.f32_to_bf16_bits(s.astype(np.float32))
    s2, n2 = P.rmsnorm(hb["sum"], sbits, hs["w2"], 1e-6)
    compare.assert_equal(hb["res"], inputs.f32_to_bf16_bits(s2.astype(np.float32)), "residual stream")
    P.assert_within(P.f64(hb["last"]), n2, P.rmsnorm_bound(n2), "second norm")


def test_decode_block_graph_replays_match_eager(dev):
    """The chain captured once and replayed with eager work on the same buffers
    in between; the captured call is not synchronised inside."""
    import torch
    import moe_glue_amd as mg

    T = 9
    st, bufs, _ = block_state(mg, torch, T, dev)
    keys = [key for key in bufs if key != "layer"]
    outs = lambda: [bufs[key] for key in keys] + [bufs["layer"][key] for key in ("topk_ids", "topk_weights", "out")]  # noqa: E731
    side = torch.cuda.Stream(device=dev)
    with torch.cuda.stream(side):
        decode_block(mg, torch, st, bufs)  # library products set themselves up outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        decode_block(mg, torch, st, bufs)
    for rep in range(4):
        other, _, _ = block_state(mg, torch, T, dev, seed=rep)
        for key in ("x", "r"):
            st[key].copy_(other[key])
        decode_block(mg, torch, st, bufs)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs()]
        for t in outs() + [bufs["layer"]["workspace"]]:
            t.view(torch.uint8).fill_(0xA5 + rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs(), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {rep}"


def test_decode_ops_on_two_streams(dev):
    """Two streams at once, each with its own buffers, calls not synchronised."""
    import torch
    import moe_glue_amd as mg

    sets = [block_state(mg, torch, T, dev, seed=T) for T in (3, 40)]
    refs = []
    for st, bufs, _ in sets:
        decode_block(mg, torch, st, bufs)
        torch.cuda.synchronize()
        refs.append((bufs["codes"].clone(), bufs["last"].clone(), bufs["layer"]["out"].clone()))
    streams = [torch.cuda.Stream(device=dev) for _ in sets]
    for _ in range(8):
        for stream, (st, bufs, _) in zip(streams, sets):
            with torch.cuda.stream(stream):
                decode_block(mg, torch, st, bufs)
    torch.cuda.synchronize()
    for (st, bufs, _), ref in zip(sets, refs):
        for got, want in zip((bufs["codes"], bufs["last"], bufs["layer"]["out"]), ref):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
