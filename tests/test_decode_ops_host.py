"""Refusals of the norm, the MXFP4 linear and the few-token layer, on the CPU:
the C ABI's status before any HIP call, and the binding's checks before any
pointer is read.  Also the 64-bit forms against hand-worked values."""
import numpy as np
import pytest

import plain64 as P
from test_boundary import FAKE, FakeGpu, lib, status  # noqa: F401

EPS = 1e-6


def test_norm_argument_errors(lib):  # noqa: F811
    def call(x=FAKE, r=None, w=FAKE, T=4, H=256, eps=EPS, ro=None, out=FAKE):
        return status(lib, lib.moe_rmsnorm(x, r, w, T, H, eps, ro, out, None))

    assert call(T=-1) == "MOE_ERR_SHAPE"
    assert call(H=0) == "MOE_ERR_SHAPE"
    assert call(H=12) == "MOE_ERR_ALIGN"
    assert call(H=65544) == "MOE_ERR_UNSUPPORTED"
    assert call(T=2 ** 31 - 1, H=65536) == "MOE_ERR_UNSUPPORTED"
    for eps in (0.0, -1e-6, float("inf"), float("nan"), 1e-39):
        assert call(eps=eps) == "MOE_ERR_UNSUPPORTED", eps
    assert call(x=None) == call(w=None) == call(out=None) == "MOE_ERR_NULL"
    assert call(ro=FAKE) == "MOE_ERR_NULL"
    assert b"residual" in lib.moe_last_error()
    for bad in ({"x": FAKE + 8}, {"w": FAKE + 8}, {"r": FAKE + 8}, {"out": FAKE + 8}, {"r": FAKE, "ro": FAKE + 8}):
        assert call(**bad) == "MOE_ERR_ALIGN", bad
    assert call(T=0, x=None, w=None, out=None) == "MOE_OK"


def test_quantised_norm_argument_errors(lib):  # noqa: F811
    def fp8(x=FAKE, T=4, H=256, group=128, q=FAKE, sc=FAKE, out=None):
        return status(lib, lib.moe_rmsnorm_fp8(x, None, FAKE, T, H, EPS, group, None, out, q, sc, None))

    for group in (0, 4, 12, 1024, -8):
        assert fp8(group=group) == "MOE_ERR_UNSUPPORTED", group
    assert fp8(H=192) == "MOE_ERR_SHAPE"
    assert fp8(q=None) == fp8(sc=None) == fp8(x=None) == "MOE_ERR_NULL"
    assert fp8(q=FAKE + 4) == fp8(sc=FAKE + 2) == fp8(out=FAKE + 8) == "MOE_ERR_ALIGN"
    assert fp8(T=0, x=None, q=None, sc=None) == "MOE_OK"

    def mx(T=4, H=256, q=FAKE, sc=FAKE):
        return status(lib, lib.moe_rmsnorm_mxfp8(FAKE, None, FAKE, T, H, EPS, None, None, q, sc, None))

    assert mx(H=48) == "MOE_ERR_SHAPE"
    assert mx(H=100) == "MOE_ERR_ALIGN"
    assert mx(q=FAKE + 4) == "MOE_ERR_ALIGN"
    assert mx(q=None) == mx(sc=None) == "MOE_ERR_NULL"
    assert mx(T=0) == "MOE_OK"


def test_decode_layer_argument_errors(lib):  # noqa: F811
    need = lib.moe_decode_layer_workspace_bytes(4, 8, 2, 64)
    assert need >= 4 * 2 * 64 * 2
    for bad in ((65, 8, 2, 64), (-1, 8, 2, 64), (4, 8, 9, 64), (4, 513, 2, 64), (4, 64, 17, 64), (4, 8, 2, 12),
                (4, 8, 2, 0), (4, 8, 2, (1 << 20) + 8)):
        assert lib.moe_decode_layer_workspace_bytes(*bad) == 0, bad

    def call(logits=FAKE, bias=None, T=4, E=8, k=2, x=FAKE, H=256, gu=FAKE, dn=FAKE, I=64, ids=FAKE, tw=FAKE, out=FAKE,
             ws=FAKE, wsb=need, mx=False, sg=FAKE, sd=FAKE):
        w = (gu, sg, dn, sd) if mx else (gu, dn)
        f = lib.moe_decode_layer_mxfp4 if mx else lib.moe_decode_layer
        return status(lib, f(logits, bias, T, E, k, x, H, *w, I, ids, tw, out, ws, wsb, None))

    for mx in (False, True):
        assert call(mx=mx, T=65) == "MOE_ERR_UNSUPPORTED"
        assert call(mx=mx, T=-1) == call(mx=mx, k=9) == call(mx=mx, k=0) == call(mx=mx, E=0) == "MOE_ERR_SHAPE"
        assert call(mx=mx, E=513) == call(mx=mx, E=64, k=17) == "MOE_ERR_UNSUPPORTED"
        assert call(mx=mx, H=0) == call(mx=mx, I=-8) == "MOE_ERR_SHAPE"
        assert call(mx=mx, H=1 << 21) == call(mx=mx, I=1 << 21) == "MOE_ERR_UNSUPPORTED"
        for key in ("logits", "x", "gu", "dn", "ids", "tw", "out"):
            assert call(mx=mx, **{key: None}) == "MOE_ERR_NULL", key
        for key in ("x", "gu", "dn", "out"):
            assert call(mx=mx, **{key: FAKE + 8}) == "MOE_ERR_ALIGN", key
        for key in ("logits", "bias", "ids", "tw"):
            assert call(mx=mx, **{key: FAKE + 2}) == "MOE_ERR_ALIGN", key
        assert call(mx=mx, wsb=need - 1) == call(mx=mx, ws=None) == call(mx=mx, ws=FAKE + 8) == "MOE_ERR_WORKSPACE"
        assert call(mx=mx, T=0, logits=None, x=None, out=None, ws=None, wsb=0) == "MOE_OK"
    assert call(H=12) == call(I=12) == "MOE_ERR_ALIGN"
    assert call(mx=True, H=48) == call(mx=True, I=48) == "MOE_ERR_SHAPE"
    assert call(mx=True, sg=None) == call(mx=True, sd=None) == "MOE_ERR_NULL"


def test_linear_argument_errors(lib):  # noqa: F811
    def call(x=FAKE, T=4, K=64, w=FAKE, sc=FAKE, N=5, y=FAKE):
        return status(lib, lib.moe_linear_mxfp4(x, T, K, w, sc, N, y, None))

    assert call(T=-1) == call(K=0) == call(N=0) == call(K=48) == "MOE_ERR_SHAPE"
    assert call(T=65) == call(K=1 << 21) == call(N=1 << 21) == "MOE_ERR_UNSUPPORTED"
    assert call(x=None) == call(w=None) == call(sc=None) == call(y=None) == "MOE_ERR_NULL"
    assert call(x=FAKE + 8) == call(w=FAKE + 8) == call(y=FAKE + 1) == "MOE_ERR_ALIGN"
    assert call(T=0, x=None, w=None, y=None) == "MOE_OK"


def _bf(*shape):
    import torch

    return FakeGpu(shape, torch.bfloat16)


def _u8(*shape):
    import torch

    return FakeGpu(shape, torch.uint8)


def _f32(*shape):
    import torch

    return FakeGpu(shape, torch.float32)


def test_binding_refuses_norm_tensors(lib):  # noqa: F811
    import moe_glue_amd as mg

    T, H = 5, 64
    x, w = _bf(T, H), _bf(H)
    with pytest.raises(ValueError, match="weight"):
        mg.rmsnorm(x, _bf(H + 8))
    with pytest.raises(ValueError, match="residual is"):
        mg.rmsnorm(x, w, _bf(T + 1, H))
    with pytest.raises(ValueError, match="residual_out without"):
        mg.rmsnorm(x, w, residual_out=_bf(T, H))
    with pytest.raises(ValueError, match="residual_out is"):
        mg.rmsnorm(x, w, _bf(T, H), residual_out=_bf(T, H - 8))
    with pytest.raises(ValueError, match="out must be"):
        mg.rmsnorm(x, w, out=_f32(T, H))
    with pytest.raises(ValueError, match="normed"):
        mg.rmsnorm_fp8(x, w, 32, normed=_bf(T, H + 8))
    for group in (0, 48, -32):
        with pytest.raises(ValueError, match="group"):
            mg.rmsnorm_fp8(x, w, group)
    with pytest.raises(ValueError, match="scales"):
        mg.rmsnorm_fp8(x, w, 32, out=_u8(T, H), scales=_f32(T, 3))
    with pytest.raises(ValueError, match="scales"):
        mg.rmsnorm_mxfp8(x, w, out=_u8(T, H), scales=_f32(T, 2))
    with pytest.raises(ValueError, match="block"):
        mg.rmsnorm_mxfp8(_bf(T, 40), _bf(40))
    import torch

    with pytest.raises(ValueError, match="GPU"):
        mg.rmsnorm(torch.zeros(2, 64, dtype=torch.bfloat16), w)


def test_binding_refuses_layer_tensors(lib):  # noqa: F811
    import torch
    import moe_glue_amd as mg

    T, E, k, H, I = 6, 8, 2, 64, 32
    logits, x, gu, dn = _f32(T, E), _bf(T, H), _bf(E, 2 * I, H), _bf(E, H, I)

    def out(**over):
        d = {"topk_ids": FakeGpu((T, k), torch.int32), "topk_weights": _f32(T, k), "out": _bf(T, H),
             "workspace": _u8(1 << 16)}
        return d | over

    call = lambda o=None, lg=logits, xx=x, a=gu, b=dn, bias=None, kk=k: mg.decode_layer(lg, kk, xx, a, b, bias=bias,  # noqa: E731
                                                                                      out=o or out())
    with pytest.raises(ValueError, match="rows"):
        call(xx=_bf(T + 1, H))
    with pytest.raises(ValueError, match="bias has"):
        call(bias=_f32(E + 1))
    for bad in (_bf(E + 1, 2 * I, H), _bf(E, 2 * I, H + 8), _bf(E, 2 * I + 1, H)):
        with pytest.raises(ValueError, match="w_gate_up"):
            call(a=bad)
    for bad in (_bf(E, H, I + 8), _bf(E - 1, H, I), _bf(E, I, H)):
        with pytest.raises(ValueError, match="w_down"):
            call(b=bad)
    for key, bad in (("topk_ids", FakeGpu((T, k + 1), torch.int32)), ("topk_weights", _f32(T * k)),
                     ("out", _bf(T, H + 8)), ("workspace", None), ("workspace", _f32(1 << 16)), ("topk_ids", None)):
        with pytest.raises(ValueError, match=key):
            call(o=out(**{key: bad}))
    for kk in (0, E + 1):
        with pytest.raises(ValueError, match="k="):
            mg.decode_layer(logits, kk, x, gu, dn)
    q = (_u8(E, 2 * I, H // 2), _u8(E, 2 * I, H // 32), _u8(E, H, I // 2), _u8(E, H, I // 32))
    for at, bad, name in ((0, _u8(E, 2 * I, H), "w_gate_up"), (1, _u8(E, 2 * I, H // 16), "s_gate_up"),
                          (2, _u8(E, H, I), "w_down"), (3, _f32(E, H, I // 32), "s_down")):
        with pytest.raises(ValueError, match=name):
            mg.decode_layer_mxfp4(logits, k, x, *(q[:at] + (bad,) + q[at + 1:]), out=out())
    with pytest.raises(ValueError, match="block"):
        mg.decode_layer_mxfp4(logits, k, _bf(T, 40), _u8(E, 2 * I, 20), q[1], _u8(E, 40, I // 2), q[3], out=out())
    other = _bf(T, H)
    other.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="cuda:0"):
        call(xx=other)


def test_binding_refuses_linear_tensors(lib):  # noqa: F811
    import moe_glue_amd as mg

    x = _bf(3, 64)
    for w, s, name in ((_u8(5, 64), _u8(5, 2), "w is"), (_u8(5, 32), _u8(5, 1), "scales"),
                       (_u8(5, 32), _u8(4, 2), "scales")):
        with pytest.raises(ValueError, match=name):
            mg.linear_mxfp4(x, w, s)
    with pytest.raises(ValueError, match="out is"):
        mg.linear_mxfp4(x, _u8(5, 32), _u8(5, 2), out=_bf(3, 4))
    with pytest.raises(ValueError, match="block"):
        mg.linear_mxfp4(_bf(3, 40), _u8(5, 20), _u8(5, 1))


def test_calls_run_with_the_tensors_device_current(lib, monkeypatch):  # noqa: F811
    """A tensor's default stream names no device of its own: the call makes the
    tensors' device current, and puts the caller's back."""
    import torch
    import moe_glue_amd as mg

    now, seen = [0], []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, now[0] = now[0], self.d.index

        def __exit__(self, *a):
            now[0] = self.old

    class Lib:
        def moe_x(self, *a):
            seen.append((now[0], a))
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(mg, "_stream", lambda d: 77 + d.index)
    monkeypatch.setattr(mg, "load", lambda: Lib())
    mg._enqueue("moe_x", torch.device("cuda", 1), 5)
    mg._enqueue("moe_x", torch.device("cuda", 0), 6)
    assert seen == [(1, (5, 78)), (0, (6, 77))] and now == [0]


# ------------------------------------------------------------- 64-bit forms
def test_plain_mxfp4_values():
    codes = np.array([[0x21, 0x43, 0x65, 0x87, 0xA9, 0xCB, 0xED, 0x0F] + [0] * 8], np.uint8)
    v = P.mxfp4_values(codes, np.array([[128]], np.uint8))[0]
    assert v[:16].tolist() == [1.0, 2.0, 3.0, 4.0, 6.0, 8.0, 12.0, -0.0, -1.0, -2.0, -3.0, -4.0, -6.0, -8.0, -12.0, 0.0]
    assert np.isnan(P.mxfp4_values(codes, np.array([[255]], np.uint8))).all()


def test_plain_e4m3_values_match_torch():
    import torch

    c = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.e4m3_values(c), t, equal_nan=True)


def test_plain_norm_and_layer_by_hand():
    one, two = 0x3F80, 0x4000
    s, n = P.rmsnorm([[one, two, one, two]], [[one, two, one, two]], [one, one, two, two], 1e-30)
    assert np.allclose(n, np.array([[2, 4, 4, 8]]) / 10 ** 0.5) and s.tolist() == [[2, 4, 2, 4]]
    # one expert, H = 2, I = 1: gate = x0, up = x1, down = (1, -3)
    out, bound = P.layer(np.array([[one, two]], np.uint16), np.array([[0]]), np.array([[0.5]]),
                         np.array([[[1.0, 0.0], [0.0, 1.0]]]), np.array([[[1.0], [-3.0]]]))
    act = 2.0 / (1.0 + np.exp(-1.0))
    assert np.allclose(out, [[0.5 * act, -1.5 * act]]) and (bound < 0.02).all()


def test_plain_route_breaks_ties_to_the_lower_expert():
    ids, w = P.route(np.array([[1.0, 3.0, 3.0, -0.0, 0.0]]), 4)
    assert ids.tolist() == [[1, 2, 0, 3]] and abs(w.sum() - 1) < 1e-15


@pytest.mark.parametrize("plant", ["swap_gate_up", "high_nibble_first", "scale_bias", "no_weight", "next_expert"])
def test_bounds_catch_planted_mistakes(plant):
    """The layer's bound is narrower than what a wrong layer is off by."""
    rng = np.random.default_rng(4)
    T, E, k, H, I = 6, 8, 2, 128, 64
    x = rng.integers(0x3E00, 0x4000, (T, H)).astype(np.uint16)
    codes = [rng.integers(0, 256, s, dtype=np.uint8) for s in ((E, 2 * I, H // 2), (E, H, I // 2))]
    scales = [rng.integers(118, 123, s, dtype=np.uint8) for s in ((E, 2 * I, H // 32), (E, H, I // 32))]
    ids, w = P.route(rng.standard_normal((T, E)), k)
    gu, dn = (P.mxfp4_values(c, s) for c, s in zip(codes, scales))
    want, bound = P.layer(x, ids, w, gu, dn)
    if plant == "swap_gate_up":
        gu = np.concatenate([gu[:, I:], gu[:, :I]], 1)
    elif plant == "high_nibble_first":
        gu = P.mxfp4_values((codes[0] >> 4) | (codes[0] << 4), scales[0])
    elif plant == "scale_bias":
        dn = P.mxfp4_values(codes[1], scales[1] + 1)
    elif plant == "no_weight":
        w = np.ones_like(w)
    else:
        ids = (ids + 1) % E
    got, _ = P.layer(x, ids, w, gu, dn)
    with pytest.raises(AssertionError):
        P.assert_within(got, want, bound, plant)
