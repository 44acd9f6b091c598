"""The experts' products (bf16, MXFP8) and their gradients on the GPU, against 64 bits:
ragged and padded segments, experts without rows, sizes round the tiles' edges, values
outside the segments that must not count."""
import pytest
import torch

import grouped64 as G

pytestmark = pytest.mark.gpu
BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
SENTINEL = 77.0


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=BF, device=g.device).normal_(0.0, std, generator=g)


def layout(ns, pad, dev, tail=0):
    """(offsets, counts or None, rows) of segments of ns rows padded to `pad`, and `tail`
    rows behind the last."""
    size = [(n + pad - 1) // pad * pad for n in ns]
    off = torch.tensor([sum(size[:e]) for e in range(len(ns) + 1)], dtype=I32, device=dev)
    return off, torch.tensor(ns, dtype=I32, device=dev) if pad > 1 else None, sum(size) + tail


def poison(t, segs, value=float("nan")):
    """Rows of no segment take `value`."""
    live = torch.zeros(t.shape[0], dtype=torch.bool, device=t.device)
    for s, n in segs:
        live[s: s + n] = True
    t[~live] = value
    return ~live


# rows: none, one, round 64, 128, 192, 256 and 320, several tiles, and more than four
RAGGED = [[0, 1, 63, 0, 64, 65], [127, 128, 129, 0], [192, 193, 255, 256, 257], [0, 0, 319, 320, 321, 1], [1100, 0, 3],
          [1], [0]]
# (the last three: enough columns for the larger tiles)
WIDTHS = [(16, 8), (64, 72), (136, 64), (264, 128), (512, 136), (528, 264), (4104, 72), (11016, 64), (11024, 136)]


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_linear(dev, case, act):
    import moe_glue_amd as mg

    g = gen(dev, 10 + case)
    ns = RAGGED[case]
    for i, (N, K) in enumerate(WIDTHS):
        N = 2 * N if act else N     # gates and ups
        pad = (1, 16, 128)[i % 3]
        off, cnt, R = layout(ns, pad, dev, tail=5)
        E = len(ns)
        x, w = normal(g, R, K), normal(g, E, N, K, std=K ** -0.5)
        bias = normal(g, E, N) if i % 2 else None
        W = N // 2 if act else N
        residual = normal(g, R, W) if i % 3 == 1 else None
        segs = G.segments(off, cnt, R)
        dead = poison(x, segs)
        out = torch.full((R, W), SENTINEL, dtype=BF, device=dev)
        pre = torch.full((R, N), SENTINEL, dtype=BF, device=dev) if act and i % 2 == 0 else None
        got = mg.grouped_linear(x, w, off, cnt, bias=bias, act=act, residual=residual, out=out, pre=pre)
        assert got is out
        what = f"{ns} N={N} K={K} pad={pad} act={act}"
        assert (out[dead] == SENTINEL).all(), f"{what}: rows of no expert were written"
        for e, (s, n) in enumerate(segs):
            want, bound, h, dh = G.linear(x[s: s + n].double(), w[e].double(), bias[e].double() if bias is not None else None,
                                          act, residual[s: s + n].double() if residual is not None else None)
            G.assert_within(out[s: s + n], want, bound, f"{what} expert {e}")
            if pre is not None:
                G.assert_within(pre[s: s + n], h, dh, f"{what} expert {e} pre")
        if pre is not None:
            assert (pre[dead] == SENTINEL).all()


@pytest.mark.parametrize("R,N,K", [(1, 8, 8), (7, 24, 4096), (16, 512, 1096), (17, 520, 640), (33, 264, 5000), (200, 2056, 328), (64, 256, 128), (65, 264, 192), (200, 1032, 520),
                                   (513, 2816, 256), (1500, 40, 64), (2048, 4104, 64)])
def test_dense(dev, R, N, K):
    """Without segments: a shared expert, its residual the very output."""
    import moe_glue_amd as mg

    g = gen(dev, R + N)
    x, w, b, r = normal(g, R, K), normal(g, N, K, std=K ** -0.5), normal(g, N), normal(g, R, N)
    want, bound, _, _ = G.linear(x.double(), w.double(), b.double(), None, r.double())
    out = r.clone()
    mg.grouped_linear(x, w, bias=b, residual=out, out=out)
    G.assert_within(out, want, bound, f"dense {R}x{N}x{K}")
    if N % 16 == 0:
        want, bound, _, _ = G.linear(x.double(), w.double(), None, "swiglu", None)
        G.assert_within(mg.grouped_linear(x, w, act="swiglu"), want, bound, f"dense swiglu {R}x{N}x{K}")


@pytest.mark.parametrize("E", [64, 65, 130, 512])
def test_many_experts(dev, E):
    """More experts than a wave has lanes, most of them without rows."""
    import moe_glue_amd as mg

    g = gen(dev, E)
    ns = [0] * E
    for i in torch.randint(0, E, (40,), generator=torch.Generator().manual_seed(E)).tolist() + [0, E - 1]:
        ns[i] += 9
    N, K = 32, 40
    for pad in (1, 16):
        off, cnt, R = layout(ns, pad, dev, tail=3)
        x, w = normal(g, R, K), normal(g, E, N, K)
        segs = G.segments(off, cnt, R)
        poison(x, segs)
        out = mg.grouped_linear(x, w, off, cnt)
        dw, db = mg.grouped_linear_grad_w(out.nan_to_num(0.0), x, off, cnt, dtype=F32, bias=True)
        for e, (s, n) in enumerate(segs):
            want, bound, _, _ = G.linear(x[s: s + n].double(), w[e].double(), None, None, None)
            G.assert_within(out[s: s + n], want, bound, f"E={E} expert {e}")
            want, bound, wb, bb = G.grad_w(out[s: s + n].double(), x[s: s + n].double(), True)
            G.assert_within(dw[e], want, bound, f"E={E} dw {e}")
            G.assert_within(db[e], wb, bb, f"E={E} db {e}")


def mx_tensor(g, *shape, low=119, high=127):
    codes = torch.randint(0, 256, shape, dtype=U8, device=g.device, generator=g)
    codes[(codes & 127) == 127] = 0
    return codes, torch.randint(low, high, (*shape[:-1], shape[-1] // 32), dtype=U8, device=g.device, generator=g)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("K", [32, 96, 128, 160, 512, 544, 1408])
def test_mxfp8(dev, K, act):
    """Scale rows of whole dwords and not (K % 128), steps that a row's end lies in."""
    import moe_glue_amd as mg

    g = gen(dev, K)
    for ns, N, pad in (([0, 1, 64, 65, 200], 48, 1), ([257, 0, 3], 272, 128), ([300], 1040, 1), ([17, 33, 65, 2], 4112, 1),
                       ([130, 193, 257, 64], 18448, 16)):
        off, cnt, R = layout(ns, pad, dev, tail=2)
        x, xs = mx_tensor(g, R, K)
        w, ws = mx_tensor(g, len(ns), N, K)
        segs = G.segments(off, cnt, R)
        poison(x, segs, 0x7F)
        poison(xs, segs, 255)
        bias = normal(g, len(ns), N)
        out = mg.grouped_linear_mxfp8(x, xs, w, ws, off, cnt, bias=bias, act=act)
        for e, (s, n) in enumerate(segs):
            want, bound, _, _ = G.linear(G.mx(x[s: s + n], xs[s: s + n]), G.mx(w[e], ws[e]), bias[e].double(), act, None,
                                         G.mx_grain(x[s: s + n], xs[s: s + n], w[e], ws[e]))
            G.assert_within(out[s: s + n], want, bound, f"K={K} {ns} expert {e}")


def test_mxfp8_unaligned_scales_and_extreme_ones(dev):
    """Scales at any byte; scale bytes 0 and 254 (2^-127, 2^127); NaN codes and scales stay
    in their row or column."""
    import moe_glue_amd as mg

    g = gen(dev, 5)
    R, N, K = 70, 40, 256
    x, xs = mx_tensor(g, R, K)
    w, ws = mx_tensor(g, N, K)
    xs[3], ws[5] = 0, 254       # the product of the two is in range, each with the others is tiny or large
    xs[4, 2] = 255
    w[7, 200] = 0x7F
    x[9, 31] = 0xFF
    raw = torch.empty(xs.numel() + ws.numel() + 8, dtype=U8, device=dev)
    a = raw[1: 1 + xs.numel()].view(xs.shape)
    b = raw[3 + xs.numel(): 3 + xs.numel() + ws.numel()].view(ws.shape)
    a.copy_(xs)
    b.copy_(ws)
    xv, wv = G.mx(x, xs), G.mx(w, ws)
    want, bound, _, _ = G.linear(xv, wv, None, None, None, G.mx_grain(x, xs, w, ws))
    # beyond bf16's range the result is infinite
    inside = want.abs() < 2.0 ** 127
    for sa, sb in ((xs, ws), (a, b)):
        out = mg.grouped_linear_mxfp8(x, sa, w, sb)
        ok = inside | torch.isnan(want)
        G.assert_within(torch.where(ok, out.double(), 0.0), torch.where(ok, want, 0.0),
                        torch.where(inside, bound, 0.0), "extreme scales")
    nan = torch.isnan(want)
    assert nan[4].all() and nan[9].all() and nan[:, 7].all() and nan.sum() == 2 * N + R - 2


def test_mxfp8_takes_what_the_expand_gives(dev):
    """The quantising expand's rows and scales in padded segments, as they lie."""
    import moe_glue_amd as mg

    g = gen(dev, 6)
    T, H, E, k, I, pad = 90, 256, 8, 2, 64, 16
    x = normal(g, T, H)
    logits = torch.empty((T, E), device=dev).normal_(generator=g)
    r = mg.route_expand_mxfp8(logits, k, x, pad_to=pad)
    w, ws = mx_tensor(g, E, 2 * I, H, low=116, high=120)
    act = mg.grouped_linear_mxfp8(r["x_expanded"], r["scales"], w, ws, r["expert_offsets"], r["expert_counts"], act="swiglu")
    assert act.shape[0] == r["x_expanded"].shape[0]
    for e, (s, n) in enumerate(G.segments(r["expert_offsets"], r["expert_counts"], act.shape[0])):
        xe, xs = r["x_expanded"][s: s + n], r["scales"][s: s + n]
        want, bound, _, _ = G.linear(G.mx(xe, xs), G.mx(w[e], ws[e]), None, "swiglu", None, G.mx_grain(xe, xs, w[e], ws[e]))
        G.assert_within(act[s: s + n], want, bound, f"expert {e}")


@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_gradients(dev, case):
    import moe_glue_amd as mg

    g = gen(dev, 30 + case)
    ns = RAGGED[case]
    for i, (N, K) in enumerate(WIDTHS + [(72, 4104), (64, 11016), (136, 11024)]):
        pad = (1, 128, 16)[i % 3]
        off, cnt, R = layout(ns, pad, dev, tail=4)
        E = len(ns)
        x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, E, N, K, std=N ** -0.5)
        segs = G.segments(off, cnt, R)
        dead = poison(x, segs)
        poison(dy, segs)
        dx = torch.full((R, K), SENTINEL, dtype=BF, device=dev)
        mg.grouped_linear_grad_x(dy, w, off, cnt, out=dx)
        assert (dx[dead] == SENTINEL).all()
        wide = i % 2 == 0
        dw, db = mg.grouped_linear_grad_w(dy, x, off, cnt, dtype=F32 if wide else BF, bias=True)
        dw2, none = mg.grouped_linear_grad_w(dy, x, off, cnt, dtype=F32 if wide else BF)
        assert none is None and torch.equal(dw, dw2), "the sums' order depends on the bias"
        what = f"{ns} N={N} K={K} pad={pad}"
        for e, (s, n) in enumerate(segs):
            dyd, xd = dy[s: s + n].double(), x[s: s + n].double()
            want, slack = G.product(dyd, w[e].double().T)
            G.assert_within(dx[s: s + n], want, G.rounded(want, slack), f"{what} dx {e}")
            want, bound, wb, bb = G.grad_w(dyd, xd, wide)
            G.assert_within(dw[e], want, bound, f"{what} dw {e}")
            G.assert_within(db[e], wb, bb, f"{what} db {e}")
            if n == 0:
                assert not dw[e].any() and not db[e].any()


@pytest.mark.parametrize("ns,N,K", [([3000, 0, 1024, 1025, 2049, 5], 64, 128), ([2500], 136, 264), ([1500, 1500], 24, 8),
                                    ([0] * 70 + [2100, 7, 4000] + [0] * 9 + [1100], 16, 40)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_in_pieces(dev, ns, N, K, wide):
    """Few tiles and many rows: the sums of an expert's pieces, joined."""
    import moe_glue_amd as mg

    g = gen(dev, N + len(ns))
    off, cnt, R = layout(ns, 16, dev, tail=1)
    x, dy = normal(g, R, K), normal(g, R, N)
    segs = G.segments(off, cnt, R)
    poison(x, segs)
    poison(dy, segs)
    need = mg.grouped_linear_grad_w_workspace_bytes(R, len(ns), N, K)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=U8, device=dev)   # NaN, and bytes behind that stay
    dw, db = mg.grouped_linear_grad_w(dy, x, off, cnt, dtype=F32 if wide else BF, bias=True, workspace=ws)
    assert (ws[need:] == 0xFF).all()
    for e, (s, n) in enumerate(segs):
        want, bound, wb, bb = G.grad_w(dy[s: s + n].double(), x[s: s + n].double(), wide)
        G.assert_within(dw[e], want, bound, f"dw {e}")
        G.assert_within(db[e], wb, bb, f"db {e}")
    again, db2 = mg.grouped_linear_grad_w(dy, x, off, cnt, dtype=F32 if wide else BF, bias=True)
    assert torch.equal(dw, again) and torch.equal(db, db2)
    with pytest.raises(ValueError, match="workspace"):
        mg.grouped_linear_grad_w(dy, x, off, cnt, workspace=ws[:need - 16])


def test_dense_gradients(dev):
    import moe_glue_amd as mg

    g = gen(dev, 9)
    for R, N, K in ((1, 8, 8), (16, 1096, 512), (17, 200, 1544), (300, 264, 520), (5000, 16, 24)):
        x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, N, K)
        want, slack = G.product(dy.double(), w.double().T)
        G.assert_within(mg.grouped_linear_grad_x(dy, w), want, G.rounded(want, slack), f"dx {R}")
        dw, db = mg.grouped_linear_grad_w(dy, x, bias=True)
        assert dw.shape == (N, K) and db.shape == (N,)
        want, bound, wb, bb = G.grad_w(dy.double(), x.double(), False)
        G.assert_within(dw, want, bound, f"dw {R}")
        G.assert_within(db, wb, bb, f"db {R}")


def test_no_rows(dev):
    import moe_glue_amd as mg

    off = torch.zeros(4, dtype=I32, device=dev)
    empty = torch.empty((0, 32), dtype=BF, device=dev)
    w = torch.ones((3, 16, 32), dtype=BF, device=dev)
    assert mg.grouped_linear(empty, w, off).shape == (0, 16)
    dy = torch.empty((0, 16), dtype=BF, device=dev)
    assert mg.grouped_linear_grad_x(dy, w, off).shape == (0, 32)
    dw = torch.full((3, 16, 32), float("nan"), dtype=BF, device=dev)
    db = torch.full((3, 16), float("nan"), device=dev)
    mg.grouped_linear_grad_w(dy, empty, off, out=dw, bias_out=db)
    assert not dw.any() and not db.any()
    # rows, but all of them nobody's
    x = torch.full((40, 32), float("nan"), dtype=BF, device=dev)
    out = torch.full((40, 16), SENTINEL, dtype=BF, device=dev)
    mg.grouped_linear(x, w, off, out=out)
    assert (out == SENTINEL).all()


def test_bad_segments_stay_inside(dev):
    """Offsets and counts outside [0, R] are taken as the nearest end; overlapping segments
    and more pieces than the workspace has room for give wrong rows and nothing else."""
    import moe_glue_amd as mg

    g = gen(dev, 3)
    R, N, K = 3000, 16, 32
    room = torch.full((3, R, K), SENTINEL, dtype=BF, device=dev)   # x between guards
    x, dy = room[1], normal(g, R, N)
    x.copy_(normal(g, R, K))
    w = normal(g, 4, N, K)
    guard = torch.full((3, R, N), SENTINEL, dtype=BF, device=dev)
    for off, cnt in (([-5, 100, 2 ** 31 - 1, -2 ** 31, 7], None), ([0, 0, 0, 0, 0], [R, R, R, R]),
                     ([2990, 5, -1, 4000, 1], [2 ** 31 - 1, -3, 20, 9])):
        off = torch.tensor(off, dtype=I32, device=dev)
        cnt = torch.tensor(cnt, dtype=I32, device=dev) if cnt is not None else None
        mg.grouped_linear(x, w, off, cnt, out=guard[1])
        assert (guard[0] == SENTINEL).all() and (guard[2] == SENTINEL).all()
        need = mg.grouped_linear_grad_w_workspace_bytes(R, 4, N, K)
        ws = torch.full((need + 4096,), 0x55, dtype=U8, device=dev)
        dw = torch.full((6, N, K), SENTINEL, dtype=F32, device=dev)
        mg.grouped_linear_grad_w(dy, x, off, cnt, out=dw[1:5], workspace=ws)
        assert (ws[need:] == 0x55).all() and (dw[0] == SENTINEL).all() and (dw[5] == SENTINEL).all()
        dx = torch.full((3, R, K), SENTINEL, dtype=BF, device=dev)
        mg.grouped_linear_grad_x(dy, w, off, cnt, out=dx[1])
        assert (dx[0] == SENTINEL).all() and (dx[2] == SENTINEL).all()
    torch.cuda.synchronize()


def test_infinities_and_nan_stay_where_they_belong(dev):
    import moe_glue_amd as mg

    g = gen(dev, 4)
    ns, N, K = [70, 130, 0, 200], 48, 96
    off, cnt, R = layout(ns, 16, dev)
    x, w = normal(g, R, K), normal(g, 4, N, K)
    x[3, 5], x[off[1] + 1, 0] = float("inf"), float("nan")
    w[3, 11, 95] = float("nan")
    out = mg.grouped_linear(x, w, off, cnt)
    for e, (s, n) in enumerate(G.segments(off, cnt, R)):
        want, bound, _, _ = G.linear(x[s: s + n].double(), w[e].double(), None, None, None)
        G.assert_within(out[s: s + n], want, bound, f"expert {e}")
    assert torch.isnan(out[off[3]: off[3] + 200, 11]).all()
    # gradients: a row's NaN reaches its expert's weight gradient alone
    dy = normal(g, R, N)
    dy[5, 7] = float("nan")
    dw, db = mg.grouped_linear_grad_w(dy, torch.ones_like(x), off, cnt, dtype=F32, bias=True)
    bad = torch.isnan(dw)
    assert bad[0, 7].all() and bad.sum() == K and torch.isnan(db).sum() == 1 and torch.isnan(db[0, 7])


def test_far_rows_and_experts(dev):
    """Byte offsets beyond 32 bits: rows of x, dy and out, experts of w and dw."""
    import moe_glue_amd as mg

    g = gen(dev, 8)
    R, K, N = 140000, 16384, 16           # x: 4.6 GB
    x = torch.zeros((R, K), dtype=BF, device=dev)
    ns = [64, R - 200, 100]
    off = torch.tensor([0, 64, R - 136, R - 36], dtype=I32, device=dev)
    x[-136:] = normal(g, 136, K)
    w = normal(g, 3, N, K, std=K ** -0.5)
    out = mg.grouped_linear(x, w, off)
    s, n = ns[0] + ns[1], ns[2]
    want, bound, _, _ = G.linear(x[s: s + n].double(), w[2].double(), None, None, None)
    G.assert_within(out[s: s + n], want, bound, "far rows")
    assert not out[64: 64 + 100].any()
    dy = torch.zeros((R, N), dtype=BF, device=dev)
    dy[s: s + n] = normal(g, n, N)
    dw, _ = mg.grouped_linear_grad_w(dy, x, off)
    want, bound, _, _ = G.grad_w(dy[s: s + n].double(), x[s: s + n].double(), False)
    G.assert_within(dw[2], want, bound, "far rows' gradient")
    dx = mg.grouped_linear_grad_x(dy, w, off)
    want, slack = G.product(dy[s: s + n].double(), w[2].double().T)
    G.assert_within(dx[s: s + n], want, G.rounded(want, slack), "far dx")
    del x, out, dy, dw, dx
    E, N, K = 300, 1024, 8192             # w: 5 GB
    w = torch.zeros((E, N, K), dtype=BF, device=dev)
    w[E - 1] = normal(g, N, K, std=K ** -0.5)
    off = torch.zeros(E + 1, dtype=I32, device=dev)
    off[E] = 70
    x = normal(g, 70, K)
    want, bound, _, _ = G.linear(x.double(), w[E - 1].double(), None, None, None)
    out = mg.grouped_linear(x, w, off)
    G.assert_within(out, want, bound, "far expert")
    dw, _ = mg.grouped_linear_grad_w(out, x, off, out=w)
    want, bound, _, _ = G.grad_w(out.double(), x.double(), False)
    G.assert_within(dw[E - 1], want, bound, "far expert's gradient")
    assert not dw[0].any() and not dw[E - 2].any()


def test_same_bits_every_time(dev):
    import moe_glue_amd as mg

    g = gen(dev, 2)
    ns, N, K = [500, 0, 77, 1300], 272, 264
    off, cnt, R = layout(ns, 1, dev)
    x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, 4, N, K)
    first = None
    for _ in range(5):
        got = (mg.grouped_linear(x, w, off, act="swiglu"), mg.grouped_linear_grad_x(dy, w, off),
               *mg.grouped_linear_grad_w(dy, x, off, bias=True))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
