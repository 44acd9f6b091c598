"""Refusals of the experts' products and the gradients, on the CPU: the C ABI's status
before any HIP call, and the binding's checks before any pointer is read.  Also the
64-bit gradients against differences of the 64-bit forward formulas."""
import pytest
import torch

import grouped64 as G
from test_boundary import FAKE, FakeGpu, lib, status  # noqa: F401

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def test_grouped_linear_argument_errors(lib):  # noqa: F811
    def call(x=FAKE, R=40, off=FAKE, cnt=None, w=FAKE, E=4, N=64, K=64, bias=None, act=0, res=None, pre=None, out=FAKE,
             mx=False, xs=FAKE, ws=FAKE):
        tail = (E, N, K, bias, act, res, pre, out, None)
        if mx:
            return status(lib, lib.moe_grouped_linear_mxfp8(x, xs, R, off, cnt, w, ws, *tail))
        return status(lib, lib.moe_grouped_linear(x, R, off, cnt, w, *tail))

    for mx in (False, True):
        assert call(mx=mx, R=-1) == call(mx=mx, E=0) == call(mx=mx, N=0) == call(mx=mx, K=0) == "MOE_ERR_SHAPE"
        assert call(mx=mx, E=513) == call(mx=mx, K=1 << 21) == call(mx=mx, N=1 << 21) == "MOE_ERR_UNSUPPORTED"
        assert call(mx=mx, R=2 ** 31 - 1, N=1 << 16) == "MOE_ERR_UNSUPPORTED"   # tiles
        assert call(mx=mx, act=2) == call(mx=mx, act=-1) == "MOE_ERR_UNSUPPORTED"
        assert call(mx=mx, N=68) == call(mx=mx, N=72, act=1) == "MOE_ERR_ALIGN"
        assert call(mx=mx, off=None) == call(mx=mx, off=None, E=1, cnt=FAKE) == "MOE_ERR_NULL"
        assert call(mx=mx, off=FAKE + 2) == call(mx=mx, cnt=FAKE + 2) == "MOE_ERR_ALIGN"
        assert call(mx=mx, pre=FAKE) == "MOE_ERR_UNSUPPORTED"
        for key in ("x", "w", "out"):
            assert call(mx=mx, **{key: None}) == "MOE_ERR_NULL", key
        for key in ("x", "w", "bias", "res", "out"):
            assert call(mx=mx, **{key: FAKE + 8}) == "MOE_ERR_ALIGN", key
        assert call(mx=mx, act=1, pre=FAKE + 8) == "MOE_ERR_ALIGN"
        assert call(mx=mx, R=0, x=None, w=None, out=None) == "MOE_OK"
    assert call(K=60) == "MOE_ERR_ALIGN"
    assert call(mx=True, K=48) == "MOE_ERR_SHAPE"
    assert call(mx=True, xs=None) == call(mx=True, ws=None) == "MOE_ERR_NULL"


def test_grouped_gradient_argument_errors(lib):  # noqa: F811
    def gx(dy=FAKE, R=40, off=FAKE, cnt=None, w=FAKE, E=4, N=64, K=64, dx=FAKE):
        return status(lib, lib.moe_grouped_linear_grad_x(dy, R, off, cnt, w, E, N, K, dx, None))

    def gw(dy=FAKE, x=FAKE, R=40, off=FAKE, cnt=None, E=4, N=64, K=64, wide=0, dw=FAKE, db=None, ws=None, wsb=0):
        return status(lib, lib.moe_grouped_linear_grad_w(dy, x, R, off, cnt, E, N, K, wide, dw, db, ws, wsb, None))

    for f in (gx, gw):
        assert f(R=-1) == f(E=0) == f(N=0) == f(K=-8) == "MOE_ERR_SHAPE"
        assert f(E=513) == f(K=1 << 21) == f(N=1 << 21) == "MOE_ERR_UNSUPPORTED"
        assert f(N=60) == f(K=60) == "MOE_ERR_ALIGN"
        assert f(off=None) == f(off=None, E=1, cnt=FAKE) == "MOE_ERR_NULL"
        assert f(off=FAKE + 2) == f(cnt=FAKE + 1) == f(dy=FAKE + 8) == "MOE_ERR_ALIGN"
        assert f(dy=None) == "MOE_ERR_NULL"
    assert gx(w=None) == gx(dx=None) == "MOE_ERR_NULL"
    assert gx(w=FAKE + 8) == gx(dx=FAKE + 8) == "MOE_ERR_ALIGN"
    assert gx(R=2 ** 31 - 1, K=1 << 16) == "MOE_ERR_UNSUPPORTED"
    assert gx(R=0, dy=None, w=None, dx=None) == "MOE_OK"
    assert gw(x=None) == gw(dw=None) == gw(R=0, dw=None) == "MOE_ERR_NULL"
    assert gw(x=FAKE + 8) == gw(dw=FAKE + 8) == gw(db=FAKE + 2) == "MOE_ERR_ALIGN"
    assert gw(E=512, N=1 << 20, K=1 << 20) == "MOE_ERR_UNSUPPORTED"
    # the workspace: for few tiles and many rows
    size = lib.moe_grouped_linear_grad_w_workspace_bytes
    assert size(40, 4, 64, 64) == 0 and size(-1, 4, 64, 64) == 0 and size(40, 4, 64, 60) == 0
    need = size(40000, 4, 64, 64)
    assert need >= 2 * 64 * 65 * 4 and need % 4 == 0
    for bad in ({"ws": None, "wsb": 0}, {"ws": FAKE, "wsb": need - 1}, {"ws": FAKE + 8, "wsb": need}):
        assert gw(R=40000, **bad) == "MOE_ERR_WORKSPACE", bad


def test_step_gradient_argument_errors(lib):  # noqa: F811
    def sw(h=FAKE, d=FAKE, R=4, I=64, dh=FAKE, act=None):
        return status(lib, lib.moe_swiglu_backward(h, d, R, I, dh, act, None))

    assert sw(R=-1) == sw(I=0) == "MOE_ERR_SHAPE"
    assert sw(I=12) == sw(h=FAKE + 8) == sw(d=FAKE + 8) == sw(dh=FAKE + 8) == sw(act=FAKE + 8) == "MOE_ERR_ALIGN"
    assert sw(R=2 ** 31 - 1, I=1024) == "MOE_ERR_UNSUPPORTED"
    assert sw(h=None) == sw(d=None) == sw(dh=None) == "MOE_ERR_NULL"
    assert sw(R=0, h=None, d=None, dh=None) == "MOE_OK"

    def cb(dout=FAKE, y=FAKE, w=FAKE, dest=FAKE, T=4, H=64, k=2, dy=FAKE, dw=FAKE):
        return status(lib, lib.moe_combine_backward(dout, y, w, dest, T, H, k, dy, dw, None))

    assert cb(T=-1) == cb(H=0) == cb(k=0) == cb(k=17) == "MOE_ERR_SHAPE"
    assert cb(T=2 ** 30, H=64) == cb(T=2 ** 28, H=8, k=16) == "MOE_ERR_UNSUPPORTED"
    for key in ("dout", "y", "dy"):
        assert cb(**{key: None}) == "MOE_ERR_NULL" and cb(**{key: FAKE + 8}) == "MOE_ERR_ALIGN", key
    for key in ("w", "dest", "dw"):
        assert cb(**{key: None}) == "MOE_ERR_NULL" and cb(**{key: FAKE + 2}) == "MOE_ERR_ALIGN", key
    assert cb(H=12) == "MOE_ERR_ALIGN"
    assert cb(T=0, dout=None, y=None, w=None, dest=None, dy=None, dw=None) == "MOE_OK"

    def eb(dxe=FAKE, dest=FAKE, res=None, T=4, H=64, k=2, dx=FAKE):
        return status(lib, lib.moe_expand_rows_backward(dxe, dest, res, T, H, k, dx, None))

    assert eb(T=-1) == eb(H=0) == eb(k=0) == eb(k=17) == "MOE_ERR_SHAPE"
    assert eb(dxe=None) == eb(dest=None) == eb(dx=None) == "MOE_ERR_NULL"
    assert eb(dxe=FAKE + 8) == eb(res=FAKE + 8) == eb(dx=FAKE + 8) == eb(dest=FAKE + 2) == eb(H=12) == "MOE_ERR_ALIGN"
    assert eb(T=0, dxe=None, dest=None, dx=None) == "MOE_OK"

    def rb(ids=FAKE, w=FAKE, dw=FAKE, T=4, E=8, k=2, dl=FAKE, db=None):
        return status(lib, lib.moe_route_backward(ids, w, dw, T, E, k, dl, db, None))

    assert rb(T=-1) == rb(E=0) == rb(k=0) == rb(k=9) == "MOE_ERR_SHAPE"
    assert rb(E=513) == rb(E=64, k=17) == "MOE_ERR_UNSUPPORTED"
    for key in ("ids", "w", "dw", "dl"):
        assert rb(**{key: None}) == "MOE_ERR_NULL" and rb(**{key: FAKE + 2}) == "MOE_ERR_ALIGN", key
    assert rb(db=FAKE + 1) == "MOE_ERR_ALIGN"
    assert rb(T=0, ids=None, w=None, dw=None, dl=None) == "MOE_OK"


def test_binding_refuses_grouped_tensors(lib):  # noqa: F811
    import moe_glue_amd as mg

    R, E, N, K = 24, 3, 32, 64
    x, w, off = FakeGpu((R, K), BF), FakeGpu((E, N, K), BF), FakeGpu((E + 1,), I32)
    with pytest.raises(ValueError, match="with offsets"):
        mg.grouped_linear(x, FakeGpu((N, K), BF), off)
    with pytest.raises(ValueError, match="without offsets"):
        mg.grouped_linear(x, w)
    with pytest.raises(ValueError, match="counts without"):
        mg.grouped_linear(x, FakeGpu((N, K), BF), counts=FakeGpu((E,), I32))
    with pytest.raises(ValueError, match="w is"):
        mg.grouped_linear(x, FakeGpu((E, N, K + 8), BF), off)
    with pytest.raises(ValueError, match="offsets is"):
        mg.grouped_linear(x, w, FakeGpu((E,), I32))
    with pytest.raises(ValueError, match="counts"):
        mg.grouped_linear(x, w, off, FakeGpu((E + 1,), I32))
    with pytest.raises(ValueError, match="bias"):
        mg.grouped_linear(x, w, off, bias=FakeGpu((E, N + 8), BF))
    with pytest.raises(ValueError, match="act="):
        mg.grouped_linear(x, w, off, act="relu")
    with pytest.raises(ValueError, match="residual is"):
        mg.grouped_linear(x, w, off, act="swiglu", residual=FakeGpu((R, N), BF))
    with pytest.raises(ValueError, match="out is"):
        mg.grouped_linear(x, w, off, out=FakeGpu((R + 1, N), BF))
    with pytest.raises(ValueError, match="pre without"):
        mg.grouped_linear(x, w, off, pre=FakeGpu((R, N), BF))
    with pytest.raises(ValueError, match="odd"):
        mg.grouped_linear(x, FakeGpu((E, 33, K), BF), off, act="swiglu")
    with pytest.raises(ValueError, match="x must be"):
        mg.grouped_linear(FakeGpu((R, K), F32), w, off)
    with pytest.raises(ValueError, match="x_scales"):
        mg.grouped_linear_mxfp8(FakeGpu((R, K), U8), None, FakeGpu((E, N, K), U8), FakeGpu((E, N, 2), U8), off)
    with pytest.raises(ValueError, match="w_scales"):
        mg.grouped_linear_mxfp8(FakeGpu((R, K), U8), FakeGpu((R, 2), U8), FakeGpu((E, N, K), U8),
                                FakeGpu((E, N, 3), U8), off)
    with pytest.raises(ValueError, match="block"):
        mg.grouped_linear_mxfp8(FakeGpu((R, 48), U8), FakeGpu((R, 1), U8), FakeGpu((E, N, 48), U8),
                                FakeGpu((E, N, 1), U8), off)
    dy = FakeGpu((R, N), BF)
    with pytest.raises(ValueError, match="w is"):
        mg.grouped_linear_grad_x(dy, FakeGpu((E, N + 8, K), BF), off)
    with pytest.raises(ValueError, match="out is"):
        mg.grouped_linear_grad_x(dy, w, off, out=FakeGpu((R, K + 8), BF))
    with pytest.raises(ValueError, match="x is"):
        mg.grouped_linear_grad_w(dy, FakeGpu((R + 1, K), BF), off)
    with pytest.raises(ValueError, match="dw must be"):
        mg.grouped_linear_grad_w(dy, x, off, dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        mg.grouped_linear_grad_w(dy, x, off, dtype=torch.float32, out=FakeGpu((E, N, K), BF))
    with pytest.raises(ValueError, match="bias_out"):
        mg.grouped_linear_grad_w(dy, x, off, out=FakeGpu((E, N, K), BF), bias_out=FakeGpu((N,), F32))
    with pytest.raises(ValueError, match="workspace"):
        mg.grouped_linear_grad_w(dy, x, off, out=FakeGpu((E, N, K), BF), workspace=FakeGpu((64,), F32))


def test_binding_refuses_step_gradient_tensors(lib):  # noqa: F811
    import moe_glue_amd as mg

    T, H, k, E = 6, 64, 2, 8
    with pytest.raises(ValueError, match="odd"):
        mg.swiglu_backward(FakeGpu((T, 33), BF), FakeGpu((T, 16), BF))
    with pytest.raises(ValueError, match="dact"):
        mg.swiglu_backward(FakeGpu((T, 32), BF), FakeGpu((T, 32), BF))
    with pytest.raises(ValueError, match="act is"):
        mg.swiglu_backward(FakeGpu((T, 32), BF), FakeGpu((T, 16), BF), out=FakeGpu((T, 32), BF), act=FakeGpu((T, 8), BF))
    dout, y, w = FakeGpu((T, H), BF), FakeGpu((T * k, H), BF), FakeGpu((T, k), F32)
    dest = FakeGpu((T * k,), I32)
    with pytest.raises(ValueError, match="at least"):
        mg.combine_backward(dout, FakeGpu((T * k - 1, H), BF), w, dest)
    with pytest.raises(ValueError, match="y is"):
        mg.combine_backward(dout, FakeGpu((T * k, H + 8), BF), w, dest)
    with pytest.raises(ValueError, match="dest_of_src"):
        mg.combine_backward(dout, y, w, FakeGpu((T,), I32))
    with pytest.raises(ValueError, match="dweights"):
        mg.combine_backward(dout, y, w, dest, out=FakeGpu((T * k, H), BF), dweights=FakeGpu((T, k + 1), F32))
    with pytest.raises(ValueError, match="multiple of k"):
        mg.expand_rows_backward(y, FakeGpu((T * k + 1,), I32), k)
    with pytest.raises(ValueError, match="at least"):
        mg.expand_rows_backward(FakeGpu((T, H), BF), dest, k)
    with pytest.raises(ValueError, match="residual"):
        mg.expand_rows_backward(y, dest, k, residual=FakeGpu((T, H + 8), BF))
    with pytest.raises(ValueError, match="topk_ids"):
        mg.route_backward(FakeGpu((T, k + 1), I32), w, w, E)
    with pytest.raises(ValueError, match="k="):
        mg.route_backward(FakeGpu((T, k), I32), w, w, 1)
    with pytest.raises(ValueError, match="bias_out"):
        mg.route_backward(FakeGpu((T, k), I32), w, w, E, out=FakeGpu((T, E), F32), bias_out=FakeGpu((E + 1,), F32))


def _along(f, at, d, eps=1e-5):
    """Central difference of the sum f along d: off by eps^2 / 6 of the third derivative and
    2^-53 / eps of f."""
    return (f(at + eps * d) - f(at - eps * d)) / (2 * eps)


def test_gradients_are_those_of_the_formulas():
    """The 64-bit gradients that the kernels are held to, against differences of the
    64-bit forward formulas (1e-6 of the magnitudes: the third derivatives are of the
    order of the values)."""
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.empty(shape, dtype=torch.float64).normal_(generator=g)

    # swiglu
    h, d, dirs = rand(7, 32), rand(7, 16), rand(7, 32)
    dh = G.swiglu_grad(h, d)[0]
    f = lambda v: (d * (v[:, :16] / (1 + torch.exp(-v[:, :16])) * v[:, 16:])).sum()  # noqa: E731
    assert abs(_along(f, h, dirs) - (dh * dirs).sum()) <= 1e-6 * (dh * dirs).abs().sum()
    # routing: weights of the selected keys, their loss <dw, w>
    T, E, k = 5, 9, 3
    logits, bias, dw = rand(T, E), rand(E), rand(T, k)
    ids = torch.topk(logits + bias, k).indices

    def weights(lo, b):
        return torch.softmax((lo + b).gather(1, ids), -1)

    dl, _, db, _ = G.route_grad(ids, weights(logits, bias), dw, E)
    dirs, dirb = rand(T, E), rand(E)
    f = lambda v: (dw * weights(v, bias)).sum()  # noqa: E731
    assert abs(_along(f, logits, dirs) - (dl * dirs).sum()) <= 1e-6 * (dl * dirs).abs().sum()
    f = lambda v: (dw * weights(logits, v)).sum()  # noqa: E731
    assert abs(_along(f, bias, dirb) - (db * dirb).sum()) <= 1e-6 * (db * dirb).abs().sum()
    # combine, expand: linear, so differences are exact but for rounding
    dest = torch.randperm(T * k, generator=g)
    y, w, dout = rand(T * k, 8), weights(logits, bias), rand(T, 8)
    comb = lambda yy, ww: (dout * (ww[:, :, None] * yy[dest.view(T, k)]).sum(1)).sum()  # noqa: E731
    dy, _, dwt, _ = G.combine_grad(dout, y, w, dest)
    dyd, wd = rand(T * k, 8), rand(T, k)
    assert abs(_along(lambda v: comb(v, w), y, dyd) - (dy.reshape(T * k, 8) * dyd[dest]).sum()) <= 1e-6
    assert abs(_along(lambda v: comb(y, v), w, wd) - (dwt * wd).sum()) <= 1e-6
    dxe, xd = rand(T * k, 8), rand(T, 8)
    dx = G.expand_grad(dxe, dest, k, None)[0]
    assert abs(_along(lambda v: (dxe[dest] * v.repeat_interleave(k, 0)).sum(), rand(T, 8), xd) - (dx * xd).sum()) <= 1e-6
    # products
    x, wt, gy = rand(6, 8), rand(16, 8), rand(6, 16)
    gw, _, gb, _ = G.grad_w(gy, x, True)
    wdir, bdir = rand(16, 8), rand(16)
    assert abs(_along(lambda v: (gy * (x @ v.T)).sum(), wt, wdir) - (gw * wdir).sum()) <= 1e-6
    assert abs(_along(lambda v: (gy * (x @ wt.T + v)).sum(), rand(16), bdir) - (gb * bdir).sum()) <= 1e-6
