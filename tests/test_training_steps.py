"""The gradients of SwiGLU, combine, expand and routing on the GPU against 64 bits, and a
training step of the whole layer, eager, on another stream and captured."""
import pytest
import torch

import grouped64 as G

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
SENTINEL = 77.0


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=BF, device=g.device).normal_(0.0, std, generator=g)


@pytest.mark.parametrize("R,I", [(1, 8), (3, 24), (257, 768), (1000, 1408), (5, 20000)])
def test_swiglu_backward(dev, R, I):
    import moe_glue_amd as mg

    g = gen(dev, R + I)
    h, d = normal(g, R, 2 * I, std=3.0), normal(g, R, I)
    want, bound, act, ab = G.swiglu_grad(h.double(), d.double())
    got_act = torch.empty((R, I), dtype=BF, device=dev)
    G.assert_within(mg.swiglu_backward(h, d, act=got_act), want, bound, "dh")
    G.assert_within(got_act, act, ab, "act")
    G.assert_within(mg.swiglu_backward(h, d), want, bound, "dh alone")
    # in place: dh over h, act over dact
    h2, d2 = h.clone(), d.clone()
    mg.swiglu_backward(h2, d2, out=h2, act=d2)
    G.assert_within(h2, want, bound, "dh over h")
    G.assert_within(d2, act, ab, "act over dact")


def test_swiglu_backward_far_gates(dev):
    """Gates from where the sigmoid is 1 to where it is below fp32, zeros of both signs,
    and infinities as the formula has them."""
    import moe_glue_amd as mg

    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1.0, -1.278, 20.0, -20.0, 80.0, -80.0, -87.0, -95.0, 200.0, -200.0, 1e30,
                      -1e30], device=dev).to(BF)
    u = torch.tensor([1.0, -3.0, 0.5, 1e-20, 100.0, 2.0, -1.0, 7.0], device=dev).to(BF)
    h = torch.cat((g.repeat_interleave(8), u.repeat(16)))[None]
    d = torch.full((1, 128), 1.5, dtype=BF, device=dev)
    want, bound, act, ab = G.swiglu_grad(h.double(), d.double())
    got_act = torch.empty((1, 128), dtype=BF, device=dev)
    G.assert_within(mg.swiglu_backward(h, d, act=got_act), want, bound, "dh")
    G.assert_within(got_act, act, ab, "act")
    h[0, 3] = float("nan")
    h[0, 128 + 5] = float("inf")
    got = mg.swiglu_backward(h, d)
    assert torch.isnan(got[0, 3]) and torch.isnan(got[0, 131])
    assert torch.isfinite(torch.cat((got[0, :3], got[0, 6:131], got[0, 132:]))).all()


def routed(g, T, E, k, pad):
    """Route outputs of random logits (the library's own), padded to `pad`."""
    import moe_glue_amd as mg

    logits = torch.empty((T, E), device=g.device).normal_(generator=g)
    return logits, (mg.route_padded(logits, k, pad) if pad > 1 else mg.route(logits, k))


def test_route_backward_same_expert_twice(dev):
    """Not what route() gives; both slots' gradients are the expert's."""
    import moe_glue_amd as mg

    ids = torch.tensor([[2, 2, 0]], dtype=I32, device=dev)
    w = torch.tensor([[0.5, 0.25, 0.25]], device=dev)
    dw = torch.tensor([[4.0, 8.0, 0.0]], device=dev)
    dl, _ = mg.route_backward(ids, w, dw, 70)     # mean 4: 0, 1, -1
    assert dl[0, 2] == 1.0 and dl[0, 0] == -1.0 and dl.abs().sum() == 2.0


@pytest.mark.parametrize("T,H,E,k,pad", [(1, 8, 1, 1, 1), (5, 64, 4, 2, 1), (33, 520, 8, 8, 16), (100, 2048, 64, 6, 128),
                                         (64, 4104, 20, 16, 1), (257, 512, 40, 9, 1), (700, 1032, 512, 3, 16)])
def test_combine_and_expand_backward(dev, T, H, E, k, pad):
    import moe_glue_amd as mg

    g = gen(dev, T + H)
    _, r = routed(g, T, E, k, pad)
    rows = r["src_of_dest"].numel()
    dest, w = r["dest_of_src"], r["topk_weights"]
    y, dout = normal(g, rows, H), normal(g, T, H)
    named = torch.zeros(rows, dtype=torch.bool, device=dev)
    named[dest.long()] = True
    y[~named] = float("nan")
    dy = torch.full((rows, H), SENTINEL, dtype=BF, device=dev)
    got, dw = mg.combine_backward(dout, y, w, dest, out=dy)
    assert (dy[~named] == SENTINEL).all(), "padding rows were written"
    want, bound, wdw, bdw = G.combine_grad(dout.double(), y.double(), w.double(), dest)
    G.assert_within(got[dest.long()].view(T, k, H), want, bound, "dy")
    G.assert_within(dw, wdw, bdw, "dweights")
    over = y.clone()   # dy over y
    _, dw2 = mg.combine_backward(dout, over, w, dest, out=over)
    assert torch.equal(over[named], dy[named]) and torch.isnan(over[~named]).all() and torch.equal(dw, dw2)

    residual = normal(g, T, H)
    want, bound = G.expand_grad(y.double(), dest, k, None)
    G.assert_within(mg.expand_rows_backward(y, dest, k), want, bound, "dx")
    want, bound = G.expand_grad(y.double(), dest, k, residual.double())
    over = residual.clone()
    mg.expand_rows_backward(y, dest, k, residual=over, out=over)
    G.assert_within(over, want, bound, "dx over its residual")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (64, 64, 6), (65, 65, 2), (1000, 128, 8), (4097, 17, 3),
                                   (300, 512, 16)])
def test_route_backward(dev, T, E, k):
    import moe_glue_amd as mg

    g = gen(dev, T + E)
    _, r = routed(g, T, E, k, 1)
    dw = torch.empty((T, k), device=dev).normal_(generator=g)
    dl = torch.full((T, E), float("nan"), device=dev)
    got, db = mg.route_backward(r["topk_ids"], r["topk_weights"], dw, E, bias=True, out=dl)
    want, bound, wb, bb = G.route_grad(r["topk_ids"], r["topk_weights"].double(), dw.double(), E)
    assert got is dl
    G.assert_within(got, want, bound, "dlogits")
    G.assert_within(db, wb, bb, "dbias")
    alone, none = mg.route_backward(r["topk_ids"], r["topk_weights"], dw, E)
    assert none is None and torch.equal(alone, dl)


def test_no_tokens(dev):
    import moe_glue_amd as mg

    e = torch.empty((0, 2), device=dev)
    ids = torch.empty((0, 2), dtype=I32, device=dev)
    db = torch.full((5,), float("nan"), device=dev)
    dl, _ = mg.route_backward(ids, e, e, 5, bias_out=db)
    assert dl.shape == (0, 5) and not db.any()
    x = torch.empty((0, 16), dtype=BF, device=dev)
    dest = torch.empty((0,), dtype=I32, device=dev)
    assert mg.expand_rows_backward(x, dest, 2).shape == (0, 16)
    dy, dw = mg.combine_backward(x, x, e, dest)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)
    assert mg.swiglu_backward(x, torch.empty((0, 8), dtype=BF, device=dev)).shape == (0, 16)


def test_ids_outside_are_passed_over(dev):
    import moe_glue_amd as mg

    ids = torch.tensor([[0, -1], [9, 2]], dtype=I32, device=dev)
    w = torch.tensor([[0.5, 0.5], [0.25, 0.75]], device=dev)
    room = torch.full((4, 4), SENTINEL, device=dev)
    mg.route_backward(ids, w, torch.tensor([[1.0, 3.0], [2.0, 6.0]], device=dev), 4, out=room[1:3])
    assert (room[0] == SENTINEL).all() and (room[3] == SENTINEL).all()
    assert room[1].tolist() == [-0.5, 0.0, 0.0, 0.0] and room[2].tolist() == [0.0, 0.0, 0.75, 0.0]


def test_far_rows(dev):
    """Byte offsets beyond 32 bits in y, dy and the expanded rows."""
    import moe_glue_amd as mg

    g = gen(dev, 1)
    T, H, k = 36000, 8192, 8          # y: 4.7 GB
    y = torch.zeros((T * k, H), dtype=BF, device=dev)
    dest = torch.arange(T * k, dtype=I32, device=dev)
    y[-2 * k:] = normal(g, 2 * k, H)
    dout = normal(g, T, H)
    w = torch.full((T, k), 1.0 / k, device=dev)
    dx = mg.expand_rows_backward(y, dest, k)
    last = torch.arange(2 * k, device=dev)
    want, bound = G.expand_grad(y[-2 * k:].double(), last, k, None)
    G.assert_within(dx[-2:], want, bound, "dx")
    want, bound, wdw, bdw = G.combine_grad(dout[-2:].double(), y[-2 * k:].double(), w[-2:].double(), last)
    dy, dw = mg.combine_backward(dout, y, w, dest, out=y)
    G.assert_within(dy[-2 * k:].view(2, k, H), want, bound, "dy")
    G.assert_within(dw[-2:], wdw, bdw, "dweights")
    assert not dw[:-2].any()


# ------------------------------------------------------------ a training step
class Layer:
    """Inputs, weights and buffers of a layer; step() is a forward and a backward pass."""

    def __init__(self, dev, seed, T=150, H=256, E=8, k=2, I=64, pad=16):
        import moe_glue_amd as mg

        g = gen(dev, seed)
        self.T, self.H, self.E, self.k, self.I, self.pad = T, H, E, k, I, pad
        self.x, self.dout = normal(g, T, H), normal(g, T, H)
        self.logits = torch.empty((T, E), device=dev).normal_(generator=g)
        self.bias = torch.empty((E,), device=dev).normal_(0, 0.5, generator=g)
        self.w1, self.b1 = normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, 2 * I, std=0.3)
        self.w2 = normal(g, E, H, I, std=I ** -0.5)
        P = mg.padded_rows(T, E, k, pad)
        self.r = mg.alloc_route_outputs(T, E, k, dev)
        self.r["src_of_dest"] = torch.empty((P,), dtype=I32, device=dev)

        def buf(*shape, dtype=BF):
            # rows of no expert hold NaN, as they may anywhere
            return torch.full(shape, float("nan"), dtype=dtype, device=dev)

        self.r["x_expanded"] = buf(P, H)
        self.h, self.act, self.y, self.out = buf(P, 2 * I), buf(P, I), buf(P, H), buf(T, H)
        self.dy, self.dact, self.dh, self.dxe, self.act2 = buf(P, H), buf(P, I), buf(P, 2 * I), buf(P, H), buf(P, I)
        self.dw, self.dlogits, self.dbias = buf(T, k, dtype=F32), buf(T, E, dtype=F32), buf(E, dtype=F32)
        self.dw1, self.db1, self.dw2 = buf(E, 2 * I, H, dtype=F32), buf(E, 2 * I, dtype=F32), buf(E, H, I)
        self.dx = buf(T, H)

    def step(self):
        import moe_glue_amd as mg

        r = mg.route_expand_padded(self.logits, self.k, self.pad, self.x, bias=self.bias, out=self.r)
        off, cnt, dest = r["expert_offsets"], r["expert_counts"], r["dest_of_src"]
        mg.grouped_linear(r["x_expanded"], self.w1, off, cnt, bias=self.b1, act="swiglu", out=self.act, pre=self.h)
        mg.grouped_linear(self.act, self.w2, off, cnt, out=self.y)
        mg.combine(self.y, r["topk_weights"], dest, out=self.out)

        mg.combine_backward(self.dout, self.y, r["topk_weights"], dest, out=self.dy, dweights=self.dw)
        mg.route_backward(r["topk_ids"], r["topk_weights"], self.dw, self.E, out=self.dlogits, bias_out=self.dbias)
        mg.grouped_linear_grad_x(self.dy, self.w2, off, cnt, out=self.dact)
        mg.swiglu_backward(self.h, self.dact, out=self.dh, act=self.act2)
        mg.grouped_linear_grad_w(self.dy, self.act2, off, cnt, out=self.dw2)
        mg.grouped_linear_grad_x(self.dh, self.w1, off, cnt, out=self.dxe)
        mg.grouped_linear_grad_w(self.dh, r["x_expanded"], off, cnt, out=self.dw1, bias_out=self.db1)
        mg.expand_rows_backward(self.dxe, dest, self.k, out=self.dx)

    RESULTS = ("out", "dx", "dlogits", "dbias", "dw1", "db1", "dw2")

    def results(self):
        return {n: getattr(self, n).clone() for n in self.RESULTS}

    def exact(self):
        """The same step in 64 bits, each expert's slots by their definition."""
        T, k, I = self.T, self.k, self.I
        key = (self.logits + self.bias).double()
        ids = self.r["topk_ids"].long()
        w = torch.softmax(key.gather(1, ids), -1)
        x, dout = self.x.double(), self.dout.double()
        got = {"out": torch.zeros_like(x), "dx": torch.zeros_like(x), "dw1": torch.zeros_like(self.dw1, dtype=torch.float64),
               "db1": torch.zeros_like(self.db1, dtype=torch.float64),
               "dw2": torch.zeros_like(self.dw2, dtype=torch.float64)}
        dwt = torch.zeros_like(w)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            w1, w2 = self.w1[e].double(), self.w2[e].double()
            h = x[t] @ w1.T + self.b1[e].double()
            gate, up = h[:, :I], h[:, I:]
            s = torch.sigmoid(gate)
            act = gate * s * up
            y = act @ w2.T
            got["out"].index_add_(0, t, w[t, j][:, None] * y)
            dwt[t, j] = (dout[t] * y).sum(-1)
            dy = w[t, j][:, None] * dout[t]
            dact = dy @ w2
            dh = torch.cat((dact * up * s * (1 + gate * (1 - s)), dact * gate * s), -1)
            got["dw2"][e], got["dw1"][e], got["db1"][e] = dy.T @ act, dh.T @ x[t], dh.sum(0)
            got["dx"].index_add_(0, t, dh @ w1)
        ds = w * (dwt - (w * dwt).sum(-1, keepdim=True))
        got["dlogits"] = torch.zeros_like(key).scatter_(1, ids, ds)
        got["dbias"] = got["dlogits"].sum(0)
        return got


def assert_near(got, want, what):
    """At most six bf16 roundings (h, act, y, dy, dact, dh) lie between inputs and any result, each
    2^-8 at most of a value whose terms add up at random: six of them in the rms are 6 * 2^-8.
    (With one expert per token dlogits and dbias are zeros, and have to be.)"""
    for n, v in want.items():
        err, size = (got[n].double() - v).pow(2).mean().sqrt(), v.pow(2).mean().sqrt()
        assert err <= 6 * G.BF16 * size, f"{what}: {n} off by {(err / size).item():.3g} in the rms"


@pytest.mark.parametrize("seed,shape", [(1, {}), (2, dict(T=1, k=1, E=3)), (3, dict(T=700, E=64, k=6, I=136, H=520, pad=1)),
                                        (4, dict(T=40, E=4, k=4, pad=128))])
def test_training_step(dev, seed, shape):
    layer = Layer(dev, seed, **shape)
    layer.step()
    assert_near(layer.results(), layer.exact(), f"{shape}")


def test_training_step_against_differences(dev):
    """<dout, out> along random directions of every input, by differences of the 64-bit
    forward pass, against the kernels' gradients.  A difference of step 1e-4 is exact to 1e-7 here; the
    gradients are off by 6 * 2^-8 in the rms of each (assert_near), which adds up at random
    along a direction of n values: sqrt(n) times that, and four times the rms is allowed."""
    layer = Layer(dev, 7, T=60, H=64, E=4, k=2, I=32)
    layer.step()
    got = layer.results()
    ids = layer.r["topk_ids"].long()
    base = {"x": layer.x.double(), "logits": layer.logits.double(), "bias": layer.bias.double(), "w1": layer.w1.double(),
            "b1": layer.b1.double(), "w2": layer.w2.double()}

    def loss(v):
        w = torch.softmax((v["logits"] + v["bias"]).gather(1, ids), -1)
        total = 0.0
        for j in range(layer.k):
            e = ids[:, j]
            h = torch.bmm(v["w1"][e], v["x"][:, :, None])[:, :, 0] + v["b1"][e]
            gate, up = h.chunk(2, -1)
            y = torch.bmm(v["w2"][e], (gate * torch.sigmoid(gate) * up)[:, :, None])[:, :, 0]
            total = total + (layer.dout.double() * w[:, j: j + 1] * y).sum()
        return total.item()

    for n, of in (("x", "dx"), ("logits", "dlogits"), ("bias", "dbias"), ("w1", "dw1"), ("b1", "db1"), ("w2", "dw2")):
        d = torch.empty_like(base[n]).normal_(generator=gen(dev, 3))
        hi, lo = dict(base), dict(base)
        hi[n], lo[n] = base[n] + 1e-4 * d, base[n] - 1e-4 * d
        want = (loss(hi) - loss(lo)) / 2e-4
        grad = got[of].double()
        allowed = 4 * 6 * G.BF16 * grad.pow(2).sum().sqrt().item() + 1e-6 * abs(want)
        assert abs((grad * d).sum().item() - want) <= allowed, n


def test_training_step_on_other_streams(dev):
    """Two layers at once on two streams, against each alone."""
    layers = [Layer(dev, s, T=400, E=16, k=4) for s in (11, 12)]
    alone = []
    for layer in layers:
        layer.step()
        alone.append(layer.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in layers]
    for _ in range(3):
        for layer, s in zip(layers, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                layer.step()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for layer, want in zip(layers, alone):
            got = layer.results()
            assert all(torch.equal(got[n], want[n]) for n in want)


def test_training_step_captured(dev):
    """The step in a graph, replayed on changing inputs with eager work between."""
    layer, other = Layer(dev, 21, T=300, E=16, k=4), Layer(dev, 21, T=300, E=16, k=4)
    layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step()
        with torch.cuda.graph(graph, stream=s):
            layer.step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        g = gen(dev, 100 + i)
        for t in (layer, other):
            g.manual_seed(100 + i)
            t.x.normal_(generator=g)
            t.dout.normal_(generator=g)
            t.logits.normal_(generator=g)
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        got, want = layer.results(), other.results()
        assert all(torch.equal(got[n], want[n]) for n in want), f"replay {i}"
