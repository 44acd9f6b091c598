"""The few-token layer and the MXFP4 linear on every path that large shapes take:
whole rounds of the loads' pipeline with a rest and a part of a step, entries of
each width, both widths of launch 2.  Each against the 64-bit form twice: within
its bound, and with the rms error of the documented roundings."""
import functools

import numpy as np
import pytest

import compare
import gpu_util as G
import plain64 as P
from moe_glue_amd import inputs


@pytest.fixture(scope="module")
def dev():
    return G.device()


def bf16(rng, shape, std=1.0):
    return inputs.f32_to_bf16_bits((std * rng.standard_normal(shape)).astype(np.float32))


def mxfp4(rng, shape, lo=118, hi=122):
    *lead, K = shape
    return (rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*lead, K // 32), dtype=np.uint8))


class Values:
    """Float64 weights, an expert at a time."""

    def __init__(self, *tensors):
        self.t = tensors
        self.shape = (*tensors[0].shape[:-1], tensors[0].shape[-1] * len(tensors))

    def __getitem__(self, e):
        return P.f64(self.t[0][e]) if len(self.t) == 1 else P.mxfp4_values(self.t[0][e], self.t[1][e])


# ---------------------------------------------------------------------- layer
@functools.lru_cache(maxsize=1)
def weights(fmt, E, H, I):
    rng = np.random.default_rng([E, H, I])
    if fmt == "bf16":
        gu, dn = (bf16(rng, (E, 2 * I, H), H ** -0.5),), (bf16(rng, (E, H, I), I ** -0.5),)
    else:
        gu, dn = mxfp4(rng, (E, 2 * I, H)), mxfp4(rng, (E, H, I))
    return gu, dn


def logits_of(kind, T, E, k, rng):
    """"even": T k / E tokens for every expert; "hot": all tokens pick expert 3 and the
    rest are even; "random"."""
    z = rng.standard_normal((T, E)).astype(np.float32)
    if kind != "random":
        pick = (np.arange(T)[:, None] * k + np.arange(k)) % E
        np.put_along_axis(z, pick, 8 + np.take_along_axis(z, pick, 1), 1)
    if kind == "hot":
        z[:, 3] += 20
    return z


# Launch 1 gives a wave all of K from 2048 (bf16) or 4096 (MXFP4) row quads on,
# entries times I / 4; a step is 128 (256) k, scales are reloaded every 2048 k.
# Launch 2 is the wide one for MXFP4 from H = 3584 on.
LAYERS = [("mxfp4", 16, 4, 3616, 1056, [(1, "random"), (8, "even"), (20, "even"), (40, "even"), (33, "hot"),
                                        (64, "hot")]),
          ("mxfp4", 16, 4, 2400, 1056, [(1, "random"), (8, "even"), (20, "even"), (40, "even"), (61, "hot")]),
          ("mxfp4", 40, 6, 4128, 416, [(1, "random"), (13, "random"), (61, "random")]),
          ("bf16", 16, 4, 1384, 520, [(1, "random"), (8, "even"), (20, "even"), (32, "even"), (48, "even"),
                                      (61, "hot"), (64, "even")]),
          ("bf16", 40, 6, 3592, 328, [(1, "random"), (13, "random"), (61, "random")])]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,E,k,H,I,T,kind", [(*s[:5], *b) for s in LAYERS for b in s[5]])
def test_layer_paths(dev, fmt, E, k, H, I, T, kind):
    import torch
    import moe_glue_amd as mg

    print(f"[layer paths] {fmt} E={E} k={k} H={H} I={I} T={T} {kind}", flush=True)
    rng = np.random.default_rng([T, E, H, len(kind)])
    logits, x = logits_of(kind, T, E, k, rng), bf16(rng, (T, H))
    gu, dn = weights(fmt, E, H, I)
    call = mg.decode_layer if fmt == "bf16" else mg.decode_layer_mxfp4
    r = call(G.to_dev(logits, dev), k, G.to_dev(x, dev), *(G.to_dev(v, dev) for v in (*gu, *dn)))
    torch.cuda.synchronize()
    ids, w = P.route(logits, k)
    compare.assert_equal(r["topk_ids"].cpu().numpy(), ids, "topk_ids")
    got = P.f64(G.to_host(r["out"]))
    want, bound = P.layer(x, ids, w, Values(*gu), Values(*dn))
    what = f"layer {fmt} {T} {kind}"
    P.assert_within(got, want, bound, what)
    P.assert_as_precise(got, *P.layer_pair(x, ids, w, Values(*gu), Values(*dn)), what)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_layer_silu_over_its_range(dev, fmt):
    """Experts that take g and u from columns 0 and 1 of x and hand act on: g from
    -3e38 to 3e38, u small and large.  silu is right to 2^-17 of its value (g log2 e
    up to 128 rounds by 2^-18, as its constant does) and 2^-118."""
    import torch
    import moe_glue_amd as mg

    T, E, k, H, I = 64, 2, 1, 32, 32
    g = np.concatenate([-np.logspace(-3, 38.4, 40), [-86, -87, -87.5, -88, -89, -100, -150, 0], np.logspace(-3, 30, 16)])
    u = np.resize([1.0, -3e7, 2e-6, 1e30, -1e-30], T)
    x = np.zeros((T, H))
    x[:, 0], x[:, 1] = g, u
    x = inputs.f32_to_bf16_bits(x.astype(np.float32))
    if fmt == "bf16":
        gu, dn = np.zeros((E, 2 * I, H), np.uint16), np.zeros((E, H, I), np.uint16)
        gu[:, 0, 0] = gu[:, I, 1] = dn[:, :, 0] = 0x3F80
        w, call = (gu, dn), mg.decode_layer
    else:
        gu, dn = np.zeros((E, 2 * I, H // 2), np.uint8), np.zeros((E, H, I // 2), np.uint8)
        gu[:, 0, 0], gu[:, I, 0], dn[:, :, 0] = 0x02, 0x20, 0x02
        one = lambda *s: np.full(s, 127, np.uint8)  # noqa: E731
        w, call = (gu, one(E, 2 * I, 1), dn, one(E, H, 1)), mg.decode_layer_mxfp4
    logits = np.zeros((T, E), np.float32)
    r = call(G.to_dev(logits, dev), k, G.to_dev(x, dev), *(G.to_dev(v, dev) for v in w))
    torch.cuda.synchronize()
    got = P.f64(G.to_host(r["out"]))
    g, u = P.f64(x[:, 0]), P.f64(x[:, 1])
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    want = silu * u
    e = (2.0 ** -17 * np.abs(silu) + 2.0 ** -118) * np.abs(u) + P.BF16_TINY
    bound = e + 2 * P.BF16 * (np.abs(want) + e) + P.BF16_TINY  # act's rounding (out's repeats it)
    fits = np.abs(want) < 3.38e38
    assert fits.sum() > 50
    P.assert_within(got[fits], np.repeat(want[fits, None], H, 1), np.repeat(bound[fits, None], H, 1), "silu")
    assert np.isinf(got[~fits]).all()


# --------------------------------------------------------------------- linear
# Every instance of both kernels; the staged one (R = 1, 2, 4 row tiles to N = 4096,
# 8192 and beyond; 16, 32 or 64 tokens) keeps 8, 4 or 2 chunks of 256 k in flight and
# gets two whole rounds of them, a rest and a part of a chunk.
LINEARS = [(17, 2336, 8195), (32, 7168, 8200), (11, 4640, 8300), (50, 1568, 8197),   # R = 4
           (13, 4640, 7001), (29, 2336, 4100), (64, 1312, 5003),                     # R = 2
           (20, 2336, 3001), (33, 1568, 4095),                                       # R = 1
           (1, 7168, 4096), (4, 4640, 8200), (8, 4640, 4099), (16, 4640, 4095), (16, 7168, 2048), (64, 4640, 2047)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", LINEARS)
def test_linear_paths(dev, T, K, N):
    import torch
    import moe_glue_amd as mg

    print(f"[linear paths] T={T} K={K} N={N}", flush=True)
    rng = np.random.default_rng([T, K, N])
    x = bf16(rng, (T, K))
    w, s = mxfp4(rng, (N, K))
    got = mg.linear_mxfp4(*(G.to_dev(v, dev) for v in (x, w, s)))
    torch.cuda.synchronize()
    got = P.f64(G.to_host(got))
    y, bound = P.linear(x, P.mxfp4_values(w, s))
    P.assert_within(got, y, bound, f"linear {T} {K} {N}")
    P.assert_as_precise(got, y, P.round_bf16(y), f"linear {T} {K} {N}")


@pytest.mark.gpu
def test_linear_scales_past_bf16(dev):
    """Under the scale bytes 253 and 254 a value beyond bf16's range is infinite, one
    inside it exact: one code a row and zeros, x = 1 on the code's column and 0 on the
    others (0 times a zero code)."""
    import torch
    import moe_glue_amd as mg

    N, K = 32, 32
    codes = np.zeros((N, K // 2), np.uint8)
    codes[:, 0] = np.arange(N) % 16
    scales = np.where(np.arange(N) < 16, 253, 254).astype(np.uint8)[:, None]
    x = np.zeros((1, K), np.uint16)
    x[0, 0] = 0x3F80
    got = P.f64(G.to_host(mg.linear_mxfp4(*(G.to_dev(v, dev) for v in (x, codes, scales)))))
    torch.cuda.synchronize()
    want = P.mxfp4_values(codes, scales)[:, 0]
    want = np.where(np.abs(want) < 2.0 ** 128, want, np.copysign(np.inf, want))
    assert np.isinf(want).any() and np.array_equal(got[0], want)


# ------------------------------------------------ what the criterion can see (CPU)
def with_significant_bits(v, n):
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 2.0 ** n) * 2.0 ** -n, e)


def model_layer(x, ids, w, gu, dn, plant):
    """The layer with fp32 products, and a mistake planted."""
    xv, I = P.f64(x), dn.shape[2]
    out = np.zeros((*ids.shape, xv.shape[1]), np.float32)
    for e in np.unique(ids):
        ts, js = np.nonzero(ids == e)
        a, wg = xv[ts].astype(np.float32), gu[e].astype(np.float32)
        if plant == "lost x column":
            a[:, -1] = 0
        h = a @ wg.T
        if plant == "bf16 h":
            h = P.round_bf16(h).astype(np.float32)
        act = h[:, :I] / (1 + np.exp(-h[:, :I])) * h[:, I:]
        act = with_significant_bits(act, 6) if plant == "6 bits of act" else P.round_bf16(act)
        if plant == "lost act column":
            act[:, -1] = 0
        y = act.astype(np.float32) @ dn[e].astype(np.float32).T
        out[ts, js] = P.round_bf16(y) if plant == "bf16 y" else y
    return P.round_bf16((w[:, :, None] * out).sum(1))


@pytest.mark.parametrize("H,I,T", [(2048, 768, 1), (1408, 264, 13)])
def test_the_criterion_sees_small_mistakes(H, I, T):
    rng = np.random.default_rng([H, T])
    E, k = 8, 4
    x, logits = bf16(rng, (T, H)), rng.standard_normal((T, E)).astype(np.float32)
    gu, dn = P.f64(bf16(rng, (E, 2 * I, H), H ** -0.5)), P.f64(bf16(rng, (E, H, I), I ** -0.5))
    ids, w = P.route(logits, k)
    pair = P.layer_pair(x, ids, w, gu, dn)
    P.assert_as_precise(model_layer(x, ids, w, gu, dn, None), *pair, "no mistake")
    for plant in ("bf16 h", "bf16 y", "6 bits of act", "lost act column", "lost x column"):
        with pytest.raises(AssertionError):
            P.assert_as_precise(model_layer(x, ids, w, gu, dn, plant), *pair, plant)


def test_round_bf16_matches_torch():
    import torch

    v = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.linspace(-140, 120, 4000),
                        [0.0, -0.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 3e38, -3.4e38]]).astype(np.float32)
    assert np.array_equal(P.round_bf16(v), torch.from_numpy(v).bfloat16().double().numpy())
