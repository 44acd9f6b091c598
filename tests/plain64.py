"""The few-token operators and the norm in 64 bits (numpy), each with a bound on
how far a correct kernel's result may be from it.

Bounds count roundings: half a step of a type is 2^-8 (bf16), 2^-24 (fp32) or
2^-4 (E4M3) of the value.  A sum of n fp32 products is off by at most
n * 2^-24 times the sum of their magnitudes for correctly rounded steps in any
order; matrix instructions may also truncate, so twice that (n * 2^-23) is
allowed.
"""
from __future__ import annotations

import numpy as np

BF16, FP32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
BF16_TINY = 2.0 ** -134   # half a step of bf16's subnormals
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def f64(bits) -> np.ndarray:
    """bf16 bits -> float64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def e4m3_values(codes) -> np.ndarray:
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def mxfp4_values(codes, scales) -> np.ndarray:
    """E2M1 codes [.., K/2] (low nibble first) and E8M0 scales [.., K/32] -> float64 [.., K]."""
    codes = np.asarray(codes, np.uint8)
    v = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    v[..., 0::2] = E2M1[codes & 15]
    v[..., 1::2] = E2M1[codes >> 4]
    s = np.where(scales == 255, np.nan, 2.0 ** (np.asarray(scales, np.float64) - 127.0))
    return v * np.repeat(s, 32, axis=-1)


def rmsnorm(x, r, w, eps):
    """(s, n) in 64 bits from bf16 bits; r may be None."""
    s = f64(x)
    if r is not None:
        s = s + f64(r)
    with np.errstate(invalid="ignore", over="ignore"):
        n = s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + np.float64(np.float32(eps))) * f64(w)
    return s, n


# Relative error of n where every step is fp32: a lane adds at most 64 squares in
# turn, then 6 lane steps and 16 waves (86 roundings, halved by the square root),
# the square's own factor s and the division, root, quotient and two products
# (7 more): 50 * 2^-24.  The kernel's steps are held to NORM_STEPS_REL below.
NORM_REL = 50 * FP32


# What the kernel's steps add up to from s = fp32(x + r) on, with its row sum,
# division and root in fp64 (2^-46 together): 1 / rms rounded and two products,
# 3 * 2^-24, and half a step for the rest.
NORM_STEPS_REL = 3.5 * FP32
FP32_TINY = 2.0 ** -149   # a step of fp32's subnormals, which n may be among


def norm_steps_bound(n) -> np.ndarray:
    """Of bf16(n)."""
    e = NORM_STEPS_REL * np.abs(n) + FP32_TINY
    return e + BF16 * (np.abs(n) + e) + BF16_TINY


def quantised_steps_bound(n, scale) -> np.ndarray:
    """Of code * scale, scale per element and as stored.  The quotient that the code
    is taken of differs from n / scale by n's steps, those of scale and of its
    inverse and the product (3 half steps): 6.5 * 2^-24; half an E4M3 step of it
    (2^-10 below its normals).  A subnormal scale is off by up to half of fp32's
    least step, 448 times in the largest code."""
    e = 7 * FP32 * np.abs(n) + 449 * FP32_TINY
    return np.maximum(E4M3 * (np.abs(n) + e), 2.0 ** -10 * scale) + e


def mx_exponent(amax) -> np.ndarray:
    """max(floor(log2 amax) - 8, -127) of float64 block maxima."""
    return np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 9, -127), -127)


def rmsnorm_bound(n) -> np.ndarray:
    return (BF16 + NORM_REL) * np.abs(n) * (1 + BF16) + BF16_TINY


def quantised_bound(n, scale) -> np.ndarray:
    """Of code * scale, scale per element: half an E4M3 step of the quotient
    (2^-10 below its normals), and n's and the scale's fp32 errors."""
    return np.maximum(E4M3 * np.abs(n), 2.0 ** -10 * scale) + 4 * NORM_REL * np.abs(n) + 2.0 ** -9 * 4 * FP32 * scale


def linear(x, w):
    """(y, bound) of x [T, K] bf16 bits times float64 weights [N, K]."""
    xv = f64(x)
    y = xv @ w.T
    slack = xv.shape[1] * 2 * FP32 * (np.abs(xv) @ np.abs(w).T)
    return y, slack + BF16 * (np.abs(y) + slack) + BF16_TINY


def route(key, k):
    """(ids, weights) of fp32 keys [T, E]: descending, equal keys to the lower expert."""
    key = np.asarray(key, np.float32) + np.float32(0.0)
    ids = np.argsort(-key.astype(np.float64), axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(key.astype(np.float64), ids, 1)
    ex = np.exp(top - top[:, :1])
    return ids.astype(np.int32), ex / ex.sum(1, keepdims=True)


def layer(x, ids, weights, wgu, wd):
    """(out, bound): x [T, H] bf16 bits, float64 weights [E, 2I, H] and [E, H, I].

    h is off by dh = H * 2^-23 * sum|x||w|; silu has slope at most 1.1, and the
    hardware's exponential and reciprocal add 2^-20 of the value; act is rounded
    to bf16; y and the sum over j add their fp32 terms, the routing weights 2^-20
    of theirs; out is rounded to bf16.
    """
    xv = f64(x)
    T, k = ids.shape
    H = xv.shape[1]
    I = wd.shape[2]
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        ts, js = np.nonzero(ids == e)
        h = xv[ts] @ wgu[e].T
        dh = H * 2 * FP32 * (np.abs(xv[ts]) @ np.abs(wgu[e]).T)
        g, u = h[:, :I], h[:, I:]
        sg = g / (1.0 + np.exp(-g))
        act = sg * u
        da = 1.1 * np.abs(u) * dh[:, :I] + (np.abs(sg) + 1.1 * dh[:, :I]) * dh[:, I:] + 2.0 ** -20 * np.abs(act)
        da = da + BF16 * (np.abs(act) + da) + BF16_TINY
        y = act @ wd[e].T
        mag = (np.abs(act) + da) @ np.abs(wd[e]).T
        dy = da @ np.abs(wd[e]).T + I * 2 * FP32 * mag
        wj = weights[ts, js][:, None]
        np.add.at(out, ts, wj * y)
        np.add.at(bound, ts, wj * (dy + (2.0 ** -20 + k * 2 * FP32) * mag))
    return out, bound + BF16 * (np.abs(out) + bound) + BF16_TINY


def round_bf16(v) -> np.ndarray:
    """Float64 -> the nearest bf16's value, through fp32 as the kernels do."""
    b = np.asarray(v, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + np.uint64(0x7FFF) + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def layer_pair(x, ids, weights, wgu, wd):
    """(exact, rounded): the layer without a rounding, and with the two that the
    calls document, of act and of out, to bf16."""
    xv = f64(x)
    exact, rounded = np.zeros(xv.shape), np.zeros(xv.shape)
    I = wd.shape[2]
    for e in np.unique(ids):
        ts, js = np.nonzero(ids == e)
        h = xv[ts] @ wgu[e].T
        act = h[:, :I] / (1.0 + np.exp(-h[:, :I])) * h[:, I:]
        wj, d = weights[ts, js][:, None], wd[e].T
        np.add.at(exact, ts, wj * (act @ d))
        np.add.at(rounded, ts, wj * (round_bf16(act) @ d))
    return exact, round_bf16(rounded)


def assert_as_precise(got, exact, rounded, what):
    """got's rms error is that of `rounded`, the exact values with the documented
    roundings.  Against those, 2^-8 at most and 2^-9.8 in the rms, fp32's own errors
    (2^-24 a step, some sqrt(K) of them) vanish, and the sums of a correct kernel
    round as the model's do but for values next to a tie: a tenth more covers it.
    One more bf16 rounding of h or y, or a lost column, adds a fifth at least."""
    got = np.asarray(got, np.float64)
    err, ref = (np.sqrt(np.mean((v - exact) ** 2)) for v in (got, rounded))
    assert err <= 1.1 * ref, f"{what}: rms error {err:.4g}, {err / ref:.2f} times that of the documented roundings"


def assert_within(got, want, bound, what):
    """|got - want| <= bound where want is finite; the same infinity or NaN elsewhere."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape} != {want.shape}"
    fine = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        bad = np.where(fine, ~(np.abs(got - want) <= bound), ~((got == want) | (np.isnan(got) & np.isnan(want))))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside, first at {i}: got {got[i]!r}, want "
                             f"{want[i]!r}, bound {np.broadcast_to(bound, want.shape)[i]!r}")
