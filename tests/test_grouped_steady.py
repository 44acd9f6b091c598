"""The experts' products in their steady state on the GPU, against 64 bits: tiles of every
height over many steps, so that each buffer is filled and read again, with a row's end inside
the last; MXFP8 with every part of the epilogue; how its sums are cut."""
import pytest
import torch

import grouped64 as G
from test_grouped import BF, SENTINEL, U8, dev, gen, layout, mx_tensor, normal, poison  # noqa: F401

pytestmark = pytest.mark.gpu
# enough columns that whole tiles are of 256 rows: 130 rows take one of 192, 193 one of 256, 257
# one of 192 and one of 128, 64 the short steps
ROWS, WIDE = [130, 193, 257, 64], 18448


def product_case(dev, K, act, N=WIDE, ns=ROWS):  # noqa: F811
    import moe_glue_amd as mg

    g = gen(dev, K)
    off, cnt, R = layout(ns, 16, dev, tail=3)
    x, w, bias = normal(g, R, K), normal(g, len(ns), N, K, std=K ** -0.5), normal(g, len(ns), N)
    W = N // 2 if act else N
    residual = normal(g, R, W)
    segs = G.segments(off, cnt, R)
    dead = poison(x, segs)
    out = torch.full((R, W), SENTINEL, dtype=BF, device=dev)
    pre = torch.full((R, N), SENTINEL, dtype=BF, device=dev) if act else None
    mg.grouped_linear(x, w, off, cnt, bias=bias, act=act, residual=residual, out=out, pre=pre)
    assert (out[dead] == SENTINEL).all()
    for e, (s, n) in enumerate(segs):
        want, bound, h, dh = G.linear(x[s: s + n].double(), w[e].double(), bias[e].double(), act,
                                      residual[s: s + n].double())
        G.assert_within(out[s: s + n], want, bound, f"K={K} N={N} expert {e}")
        if act:
            G.assert_within(pre[s: s + n], h, dh, f"K={K} N={N} expert {e} pre")
    again = torch.full_like(out, SENTINEL)
    mg.grouped_linear(x, w, off, cnt, bias=bias, act=act, residual=residual, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("K", [520, 1096, 2048])
def test_linear(dev, K, act):  # noqa: F811
    """9, 18 (both with a row's end in the last) and 32 steps of 64 columns."""
    product_case(dev, K, act)


@pytest.mark.parametrize("ns,N", [(ROWS, 11016), ([70, 128, 1, 64], 5528)])
def test_linear_lower_tiles(dev, ns, N):  # noqa: F811
    """Tiles of up to 128 and up to 64 rows."""
    product_case(dev, 1096, None, N, ns)
    product_case(dev, 1096, "swiglu", 2 * N // 16 * 16, ns)


@pytest.mark.parametrize("N", [520, 1096, 2048])
def test_grad_x(dev, N):  # noqa: F811
    """The sum runs over the weights' rows, so dx has the many columns."""
    import moe_glue_amd as mg

    g = gen(dev, N)
    off, cnt, R = layout(ROWS, 16, dev, tail=3)
    dy, w = normal(g, R, N), normal(g, len(ROWS), N, WIDE, std=N ** -0.5)
    segs = G.segments(off, cnt, R)
    dead = poison(dy, segs)
    dx = torch.full((R, WIDE), SENTINEL, dtype=BF, device=dev)
    mg.grouped_linear_grad_x(dy, w, off, cnt, out=dx)
    assert (dx[dead] == SENTINEL).all()
    for e, (s, n) in enumerate(segs):
        want, slack = G.product(dy[s: s + n].double(), w[e].double().T)
        G.assert_within(dx[s: s + n], want, G.rounded(want, slack), f"N={N} expert {e}")
    assert torch.equal(dx[~dead], mg.grouped_linear_grad_x(dy, w, off, cnt)[~dead])


# few tiles (each height of them), tiles of 64 rows, and tiles of 256
@pytest.mark.parametrize("ns,N", [([5, 0, 17, 40], 48), ([60, 64, 3], 5520), (ROWS, WIDE)])
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("K", [640, 1120])
def test_mxfp8_with_residual_and_pre(dev, ns, N, act, K):  # noqa: F811
    """Bias, residual (once the very output) and the rows before the activation; scale rows of
    whole dwords and not."""
    import moe_glue_amd as mg

    g = gen(dev, K + N)
    off, cnt, R = layout(ns, 16, dev, tail=2)
    x, xs = mx_tensor(g, R, K)
    w, ws = mx_tensor(g, len(ns), N, K)
    segs = G.segments(off, cnt, R)
    dead = poison(x, segs, 0x7F)
    poison(xs, segs, 255)
    W = N // 2 if act else N
    # of the products' own size, so that neither hides the other
    bias, residual = normal(g, len(ns), N, std=4000.0), normal(g, R, W, std=4000.0)
    pre = torch.full((R, N), SENTINEL, dtype=BF, device=dev) if act else None
    out = residual.clone()
    mg.grouped_linear_mxfp8(x, xs, w, ws, off, cnt, bias=bias, act=act, residual=out, out=out, pre=pre)
    assert torch.equal(out[dead], residual[dead])
    for e, (s, n) in enumerate(segs):
        if n == 0:
            continue
        a, b = (x[s: s + n], xs[s: s + n]), (w[e], ws[e])
        want, bound, h, dh = G.linear(G.mx(*a), G.mx(*b), bias[e].double(), act, residual[s: s + n].double(),
                                      G.mx_grain(*a, *b))
        G.assert_within(out[s: s + n], want, bound, f"K={K} N={N} expert {e}")
        if act:
            G.assert_within(pre[s: s + n], h, dh, f"K={K} N={N} expert {e} pre")
    again = mg.grouped_linear_mxfp8(x, xs, w, ws, off, cnt, bias=bias, act=act, residual=residual)
    assert torch.equal(out[~dead], again[~dead])


@pytest.mark.parametrize("R,N", [(3, 8), (70, 18440)])
def test_bf16_sums_keep_24_bits(dev, R, N):  # noqa: F811
    """2^16 - 2^16 + 2^j, which fp32 sums hold in any order down to j = -7 (2^16 + 2^-7 has 24
    bits)."""
    import moe_glue_amd as mg

    for j in range(15, -8, -1):
        for at in (23, 200):
            x, w = torch.zeros((R, 256), dtype=BF, device=dev), torch.zeros((N, 256), dtype=BF, device=dev)
            x[:, 16], x[:, 17], w[:, 16:18] = 256.0, -256.0, 256.0
            x[:, at], w[:, at] = 1.0, 2.0 ** j
            out = mg.grouped_linear(x, w).double()
            assert (out == 2.0 ** j).all(), (j, at, out[0, 0].item())


@pytest.mark.parametrize("R,N", [(3, 8), (70, 18440)])
def test_mxfp8_sums_keep_what_the_header_says(dev, R, N):  # noqa: F811
    """2^16 - 2^16 + 2^j: among eight neighbours 2^j is kept from 2^3 on (13 bits below 2^16) and
    off by no more than itself below; in different eights it is kept whole."""
    import moe_glue_amd as mg

    def code(v):
        return int(torch.tensor(v).to(torch.float8_e4m3fn).view(U8))

    K = 256
    one = torch.full((N, K // 32), 127, dtype=U8, device=dev)
    for j in range(15, -9, -1):
        a, b = (j + 1) // 2, j // 2                 # 2^j = 2^a 2^b, both E4M3 values
        for far in (False, True):
            x = torch.zeros((R, K), dtype=U8, device=dev)
            w = torch.zeros((N, K), dtype=U8, device=dev)
            x[:, 16], w[:, 16] = code(256.0), code(256.0)
            x[:, 17], w[:, 17] = code(-256.0), code(256.0)
            at = 200 if far else 23
            x[:, at], w[:, at] = code(2.0 ** a), code(2.0 ** b)
            out = mg.grouped_linear_mxfp8(x, one[:1].expand(R, -1).contiguous(), w, one).double()
            if far or j >= 3:
                assert (out == 2.0 ** j).all(), (j, far, out[0, 0].item())
            else:
                assert ((out >= 0) & (out <= 2.0 ** j)).all(), (j, far, out[0, 0].item())
