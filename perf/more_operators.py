"""The experts' products and the training side of moe_glue, case by case: products of expert-contiguous rows with the
experts' weights (bias, SwiGLU and residual in the epilogue; bf16 or MXFP8), their gradients, SwiGLU's gradient, and
the gradients of dispatch, combine and routing.

A case is run in its plain form, in elementary torch operations in fp32, or (``own``) by the library's calls.  Rows
that belong to no expert (padding, and those behind the last segment) are left as they were, zeros here."""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # ---- products of rows in expert order: out = act(x W_e^T + b_e) + residual
        # the tiny workload's gate and up rows (16 tokens, 2 experts each): launch latency
        {"name": "linear tiny", "op": "linear", "fmt": "bf16", "R": 32, "E": 8, "N": 256, "K": 256, "act": "swiglu",
         "bias": False, "residual": False, "pre": False, "pad": 1, "zipf": 0.0},
        # the benchmark's prefill batch at the Qwen3-30B-A3B shape, gate and up rows (4096 tokens, 8 experts each)
        {"name": "linear prefill", "op": "linear", "fmt": "bf16", "R": 32768, "E": 128, "N": 1536, "K": 2048,
         "act": "swiglu", "bias": False, "residual": False, "pre": False, "pad": 1, "zipf": 0.0},
        # a shared expert (no segments) of the skewed workload in training: gate and up rows with a bias, the rows
        # before the activation kept for the backward pass; an odd batch
        {"name": "linear shared odd", "op": "linear", "fmt": "bf16", "R": 1023, "E": 0, "N": 2816, "K": 4096,
         "act": "swiglu", "bias": True, "residual": False, "pre": True, "pad": 1, "zipf": 0.0},
        # a shared expert's down rows at the DeepSeek-V3 shape, added to what the routed experts gave
        {"name": "linear shared large", "op": "linear", "fmt": "bf16", "R": 8192, "E": 0, "N": 7168, "K": 2048,
         "act": "none", "bias": False, "residual": True, "pre": False, "pad": 1, "zipf": 0.0},
        # MXFP8 rows as the quantising expand lays them out, segments padded to 128 rows, skewed routing (1023 tokens,
        # 6 experts each)
        {"name": "linear mxfp8 skewed", "op": "linear", "fmt": "mxfp8", "R": 6138, "E": 64, "N": 2816, "K": 4096,
         "act": "swiglu", "bias": False, "residual": False, "pre": False, "pad": 128, "zipf": 1.2},
        # MXFP8 experts over the prefill batch
        {"name": "linear mxfp8 prefill", "op": "linear", "fmt": "mxfp8", "R": 32768, "E": 128, "N": 1536, "K": 2048,
         "act": "swiglu", "bias": False, "residual": False, "pre": False, "pad": 1, "zipf": 0.0},
        # ---- gradients of those products, to the rows, the weights and the bias
        # skewed routing, padded segments, fp32 weight gradients: some experts have most rows, some few
        {"name": "linear grad skewed", "op": "linear_grad", "R": 6138, "E": 64, "N": 4096, "K": 1408, "bias": True,
         "wide": True, "pad": 128, "zipf": 1.2},
        # the prefill batch as a training batch, gate and up rows
        {"name": "linear grad prefill", "op": "linear_grad", "R": 32768, "E": 128, "N": 1536, "K": 2048,
         "bias": False, "wide": False, "pad": 1, "zipf": 0.0},
        # ---- SwiGLU's gradient
        # the decode workload's rows (32 tokens, 8 experts each): a small step
        {"name": "swiglu grad small", "op": "swiglu_grad", "R": 256, "I": 768, "act": False},
        # the prefill batch, the activation computed again for the down rows' weight gradient
        {"name": "swiglu grad prefill", "op": "swiglu_grad", "R": 32768, "I": 768, "act": True},
        # ---- gradients of combine, routing and dispatch
        # the skewed workload with the router bias; an odd batch
        {"name": "dispatch grad odd", "op": "dispatch_grad", "T": 1023, "H": 4096, "E": 64, "k": 6, "bias": True,
         "residual": False, "pad": 1, "zipf": 1.2},
        # the DeepSeek-V3 batch: most bytes; the skip connection's gradient added to the rows'
        {"name": "dispatch grad large", "op": "dispatch_grad", "T": 8192, "H": 7168, "E": 256, "k": 8, "bias": False,
         "residual": True, "pad": 1, "zipf": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear", "linear_grad", "linear_grad", "swiglu_grad", "dispatch_grad"))
    if op == "swiglu_grad":
        while True:
            c = {"op": op, "R": _log(rng, 1, 65536), "I": 8 * _log(rng, 8, 512), "act": rng.random() < 0.5}
            if c["R"] * c["I"] <= 32768 * 768:
                return c
    if op == "dispatch_grad":
        while True:
            E = _log(rng, 2, 256)
            c = {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 1024), "E": E,
                 "k": rng.randint(1, min(E, 12)), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5,
                 "pad": rng.choice((1, 1, 16, 128)), "zipf": rng.choice((0.0, 0.0, 1.2))}
            if c["T"] * c["H"] * c["k"] <= 8192 * 7168 * 8:
                return c
    while True:
        fmt = rng.choice(("bf16", "bf16", "mxfp8")) if op == "linear" else "bf16"
        unit = 32 if fmt == "mxfp8" else 8
        E = rng.choice((0, _log(rng, 1, 256), _log(rng, 1, 256)))
        R = _log(rng, 1, 32768)
        act = rng.choice(("none", "swiglu"))
        N, K = 16 * _log(rng, 4, 448), unit * _log(rng, 128 // unit, 7168 // unit)
        if R * N * K > 32768 * 1536 * 2048 or max(E, 1) * N * K > 128 * 1536 * 2048 or R * (N + K) > 32768 * 3584:
            continue
        c = {"op": op, "R": R, "E": E, "N": N, "K": K, "bias": rng.random() < 0.4,
             "pad": 1 if E == 0 else rng.choice((1, 1, 16, 128)), "zipf": rng.choice((0.0, 0.0, 1.2))}
        if op == "linear_grad":
            c["wide"] = rng.random() < 0.4
        else:
            c.update({"fmt": fmt, "act": act, "residual": rng.random() < 0.3,
                      "pre": act == "swiglu" and rng.random() < 0.4})
        return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, std, g):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _logits(T, E, zipf, g):
    logits = torch.empty((T, E), device="cuda").normal_(generator=g)
    if zipf > 0.0:
        rank = torch.randperm(E, device="cuda", generator=g) + 1
        logits = logits - zipf * torch.log(rank.float())
    return logits


def _segments(counts, pad):
    """Offsets [E+1] of segments padded to `pad` rows."""
    off = torch.zeros(counts.numel() + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum((counts + pad - 1) // pad * pad, 0)
    return off


def _mxfp8(shape, std, g, live=None):
    """E4M3 codes and E8M0 scale bytes per 32 columns of normal values (0 outside `live` rows)."""
    v = torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).unflatten(-1, (-1, 32))
    e = torch.frexp(v.abs().amax(-1)).exponent - 9
    codes = torch.ldexp(v, -e[..., None]).clamp(-448.0, 448.0).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (e + 127).to(torch.uint8)
    if live is not None:
        codes, scales = codes * live[:, None], scales * live[:, None]
    return codes, scales


def _rows_of(c, g):
    """Segments of R rows routed to E experts; the buffers' rows; which rows are some expert's."""
    E, R = c["E"], c["R"]
    if E == 0:
        c["offsets"] = c["counts"] = None
        c["segs"] = [(0, R)]
        c["rows"] = R
        c["live"] = torch.ones(R, dtype=torch.uint8, device="cuda")
        return
    # each row's expert; all of one token's k rows differ in earnest, which changes no size
    counts = torch.bincount(_logits(R, E, c["zipf"], g).argmax(-1), minlength=E).int()
    off = _segments(counts, c["pad"])
    c["offsets"], c["counts"] = off, counts if c["pad"] > 1 else None
    starts, ns = off.tolist(), counts.tolist()
    c["segs"] = list(zip(starts, ns))
    c["rows"] = R + E * (c["pad"] - 1)  # what a program allocates before it knows the counts
    live = torch.zeros(c["rows"], dtype=torch.uint8, device="cuda")
    for s, n in c["segs"]:
        live[s: s + n] = 1
    c["live"] = live


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "swiglu_grad":
        R, I = c["R"], c["I"]
        c["h"], c["dact"] = _normal((R, 2 * I), 1.0, g), _normal((R, I), 1.0, g)
        c["dh"] = torch.empty_like(c["h"])
        c["act_out"] = torch.empty_like(c["dact"]) if c["act"] else None
        return c
    if c["op"] == "dispatch_grad":
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        top, ids = torch.sort(_logits(T, E, c["zipf"], g), dim=-1, descending=True, stable=True)
        c["ids"] = ids[:, :k].int().contiguous()
        c["weights"] = torch.softmax(top[:, :k], -1)
        flat = c["ids"].flatten().long()
        counts = torch.bincount(flat, minlength=E)
        off = _segments(counts, c["pad"])
        order = torch.argsort(flat, stable=True)
        first = torch.cumsum(counts, 0) - counts
        dest = torch.empty(T * k, dtype=torch.int32, device="cuda")
        sorted_e = flat[order]
        dest[order] = (off[sorted_e] + (torch.arange(T * k, device="cuda") - first[sorted_e])).int()
        c["dest"] = dest
        rows = T * k + E * (c["pad"] - 1)
        c["dout"], c["y"] = _normal((T, H), 1.0, g), _normal((rows, H), 1.0, g)
        c["dxe"] = _normal((rows, H), 1.0, g)
        c["dres"] = _normal((T, H), 1.0, g) if c["residual"] else None
        c["dy"] = torch.zeros_like(c["y"])
        c["dweights"] = torch.empty((T, k), device="cuda")
        c["dlogits"] = torch.empty((T, E), device="cuda")
        c["dbias"] = torch.empty((E,), device="cuda") if c["bias"] else None
        c["dx"] = torch.empty_like(c["dout"])
        return c
    _rows_of(c, g)
    N, K, rows = c["N"], c["K"], c["rows"]
    shape = (c["E"], N, K) if c["E"] else (N, K)
    live = c["live"][:, None]
    if c["op"] == "linear_grad":
        c["x"], c["dy"] = _normal((rows, K), 1.0, g) * live, _normal((rows, N), 1.0, g) * live
        c["w"] = _normal(shape, 0.02, g)
        c["dx"] = torch.zeros_like(c["x"])
        c["dw"] = torch.empty(shape, dtype=torch.float32 if c["wide"] else torch.bfloat16, device="cuda")
        c["db"] = torch.empty(shape[:-1], device="cuda") if c["bias"] else None
        return c
    if c["fmt"] == "bf16":
        c["x"], c["w"] = _normal((rows, K), 1.0, g) * live, _normal(shape, 0.02, g)
    else:
        c["x"], c["xs"] = _mxfp8((rows, K), 1.0, g, c["live"])
        c["w"], c["ws"] = _mxfp8(shape, 0.02, g)
    out_w = N // 2 if c["act"] == "swiglu" else N
    c["b"] = _normal(shape[:-1], 0.5, g) if c["bias"] else None
    c["r"] = _normal((rows, out_w), 1.0, g) if c["residual"] else None
    c["out"] = torch.zeros((rows, out_w), dtype=torch.bfloat16, device="cuda")
    c["pre_out"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda") if c["pre"] else None
    return c


# --------------------------------------------------------------- plain forms
def _mx_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)


def _expert(t, e, dense):
    return t if dense else t[e]


def _plain_linear(c):
    dense = c["E"] == 0
    out = torch.zeros_like(c["out"])
    pre = torch.zeros_like(c["pre_out"]) if c["pre"] else None
    for e, (s, n) in enumerate(c["segs"]):
        if n == 0:
            continue
        w = _expert(c["w"], e, dense)
        if c["fmt"] == "bf16":
            h = c["x"][s: s + n].float() @ w.float().T
        else:
            h = _mx_values(c["x"][s: s + n], c["xs"][s: s + n]) @ _mx_values(w, _expert(c["ws"], e, dense)).T
        if c["bias"]:
            h = h + _expert(c["b"], e, dense).float()
        if pre is not None:
            pre[s: s + n] = h
        if c["act"] == "swiglu":
            gate, up = h.chunk(2, -1)
            h = gate / (1.0 + torch.exp(-gate)) * up
        if c["residual"]:
            h = h + c["r"][s: s + n].float()
        out[s: s + n] = h
    return {"out": out, "pre": pre} if c["pre"] else {"out": out}


def _plain_linear_grad(c):
    dense = c["E"] == 0
    dx = torch.zeros_like(c["dx"])
    dw = torch.zeros_like(c["dw"])
    db = torch.zeros_like(c["db"]) if c["bias"] else None
    for e, (s, n) in enumerate(c["segs"]):
        if n == 0:
            continue
        dy = c["dy"][s: s + n].float()
        dx[s: s + n] = dy @ _expert(c["w"], e, dense).float()
        _expert(dw, e, dense).copy_(dy.T @ c["x"][s: s + n].float())
        if c["bias"]:
            _expert(db, e, dense).copy_(dy.sum(0))
    return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}


def _plain_swiglu_grad(c):
    gate, up = c["h"].float().chunk(2, -1)
    d = c["dact"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dh = torch.cat((d * up * sig * (1.0 + gate * (1.0 - sig)), d * gate * sig), -1).to(torch.bfloat16)
    return {"dh": dh, "act": (gate * sig * up).to(torch.bfloat16)} if c["act"] else {"dh": dh}


def _plain_dispatch_grad(c):
    T, H, k = c["T"], c["H"], c["k"]
    dest = c["dest"].long()
    dy = torch.zeros_like(c["dy"])
    dw = torch.empty_like(c["dweights"])
    dx = c["dres"].float() if c["residual"] else torch.zeros((T, H), device="cuda")
    dout = c["dout"].float()
    for j in range(k):
        at = dest[j::k]
        dw[:, j] = (dout * c["y"][at].float()).sum(-1)
        dy[at] = (c["weights"][:, j: j + 1] * dout).to(torch.bfloat16)
        dx = dx + c["dxe"][at].float()
    w = c["weights"]
    ds = w * (dw - (w * dw).sum(-1, keepdim=True))
    dlogits = torch.zeros((T, c["E"]), device="cuda").scatter_(1, c["ids"].long(), ds)
    got = {"dy": dy, "dweights": dw, "dlogits": dlogits, "dx": dx.to(torch.bfloat16)}
    if c["bias"]:
        got["dbias"] = dlogits.sum(0)
    return got


# --------------------------------------------------------- the library's calls
def _own_linear(c):
    import moe_glue_amd as mg

    act = None if c["act"] == "none" else c["act"]
    if c["fmt"] == "bf16":
        out = mg.grouped_linear(c["x"], c["w"], c["offsets"], c["counts"], bias=c["b"], act=act, residual=c["r"],
                                out=c["out"], pre=c["pre_out"])
    else:
        out = mg.grouped_linear_mxfp8(c["x"], c["xs"], c["w"], c["ws"], c["offsets"], c["counts"], bias=c["b"],
                                      act=act, residual=c["r"], out=c["out"], pre=c["pre_out"])
    return {"out": out, "pre": c["pre_out"]} if c["pre"] else {"out": out}


def _own_linear_grad(c):
    import moe_glue_amd as mg

    dx = mg.grouped_linear_grad_x(c["dy"], c["w"], c["offsets"], c["counts"], out=c["dx"])
    dw, db = mg.grouped_linear_grad_w(c["dy"], c["x"], c["offsets"], c["counts"], out=c["dw"], bias_out=c["db"])
    return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}


def _own_swiglu_grad(c):
    import moe_glue_amd as mg

    dh = mg.swiglu_backward(c["h"], c["dact"], out=c["dh"], act=c["act_out"])
    return {"dh": dh, "act": c["act_out"]} if c["act"] else {"dh": dh}


def _own_dispatch_grad(c):
    import moe_glue_amd as mg

    dy, dw = mg.combine_backward(c["dout"], c["y"], c["weights"], c["dest"], out=c["dy"], dweights=c["dweights"])
    dlogits, dbias = mg.route_backward(c["ids"], c["weights"], dw, c["E"], out=c["dlogits"], bias_out=c["dbias"])
    dx = mg.expand_rows_backward(c["dxe"], c["dest"], c["k"], residual=c["dres"], out=c["dx"])
    got = {"dy": dy, "dweights": dw, "dlogits": dlogits, "dx": dx}
    if c["bias"]:
        got["dbias"] = dbias
    return got


def run(state):
    op = state["op"]
    if own:
        return {"linear": _own_linear, "linear_grad": _own_linear_grad, "swiglu_grad": _own_swiglu_grad,
                "dispatch_grad": _own_dispatch_grad}[op](state)
    return {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "swiglu_grad": _plain_swiglu_grad,
            "dispatch_grad": _plain_dispatch_grad}[op](state)


# --------------------------------------------------------------------- work
def _active(c):
    """Experts with a row: a simulated batch of the case's distribution."""
    E, R = c["E"], c["R"]
    if E == 0:
        return 1
    z = np.random.default_rng(1).standard_normal((R, E), dtype=np.float32)
    if c["zipf"] > 0.0:
        z -= c["zipf"] * np.log(np.arange(1, E + 1, dtype=np.float32))
    return np.unique(z.argmax(1)).size


def work(case):
    if case["op"] == "swiglu_grad":
        n = case["R"] * case["I"]
        return {"bytes": 2 * n * (5 + (1 if case["act"] else 0)), "flops": 12 * n}
    if case["op"] == "dispatch_grad":
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        rows = T * H * 2
        return {"bytes": rows * (2 + 3 * k + (1 if case["residual"] else 0)) + T * k * 20 + T * E * 4,
                "flops": T * H * k * 4}
    R, N, K = case["R"], case["N"], case["K"]
    n_exp = max(case["E"], 1)
    if case["op"] == "linear_grad":
        # every expert's weight gradient is written, with or without rows
        return {"bytes": 2 * _active(case) * N * K + n_exp * N * K * (4 if case["wide"] else 2)
                + 2 * R * (N + 2 * K) + (4 * n_exp * N if case["bias"] else 0),
                "flops": 4 * R * N * K}
    per = 2.0 if case["fmt"] == "bf16" else 1.0 + 1 / 32
    out_w = N // 2 if case["act"] == "swiglu" else N
    return {"bytes": per * (_active(case) * N * K + R * K)
            + 2 * R * (out_w * (2 if case["residual"] else 1) + (N if case["pre"] else 0)),
            "flops": 2 * R * N * K}


# ------------------------------------------------------------- 64-bit values
def _e4m3_f64(codes):
    """Values from the format's fields: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    b = codes.double()
    sign = torch.where(b >= 128, -1.0, 1.0)
    b = b - 128.0 * (b >= 128)
    ex, m = torch.floor(b / 8), b % 8
    return sign * torch.where(ex == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (ex - 10))


def _mx_f64(codes, scales):
    return _e4m3_f64(codes) * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)


def _exact_linear(c):
    got = {"out": torch.zeros(c["out"].shape, dtype=torch.float64, device="cuda")}
    if c["pre"]:
        got["pre"] = torch.zeros(c["pre_out"].shape, dtype=torch.float64, device="cuda")
    I = c["N"] // 2
    for e, (s, n) in enumerate(c["segs"]):
        if n == 0:
            continue
        at = slice(s, s + n)
        pick = (lambda t: t[e]) if c["E"] else (lambda t: t)
        if c["fmt"] == "bf16":
            h = torch.matmul(c["x"][at].double(), pick(c["w"]).double().T)
        else:
            h = torch.matmul(_mx_f64(c["x"][at], c["xs"][at]), _mx_f64(pick(c["w"]), pick(c["ws"])).T)
        if c["bias"]:
            h += pick(c["b"]).double()
        if c["pre"]:
            got["pre"][at] = h
        if c["act"] == "swiglu":
            h = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        got["out"][at] = h + c["r"][at].double() if c["residual"] else h
    return got


def _exact_linear_grad(c):
    dx = torch.zeros(c["dx"].shape, dtype=torch.float64, device="cuda")
    dw, db = [], []
    for e, (s, n) in enumerate(c["segs"]):
        dy, x = c["dy"][s: s + n].double(), c["x"][s: s + n].double()
        dx[s: s + n] = torch.matmul(dy, (c["w"][e] if c["E"] else c["w"]).double())
        dw.append(torch.matmul(dy.T, x))
        db.append(dy.T @ torch.ones(n, dtype=torch.float64, device="cuda"))
    got = {"dx": dx, "dw": torch.stack(dw) if c["E"] else dw[0]}
    if c["bias"]:
        got["db"] = torch.stack(db) if c["E"] else db[0]
    return got


def _exact_swiglu_grad(c):
    I = c["I"]
    g, u, d = c["h"][:, :I].double(), c["h"][:, I:].double(), c["dact"].double()
    s = torch.sigmoid(g)
    silu = g * s
    got = {"dh": torch.cat((d * u * (s + silu * (1 - s)), d * silu), 1)}
    if c["act"]:
        got["act"] = silu * u
    return got


def _exact_dispatch_grad(c):
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    dest = c["dest"].long().view(T, k)
    w = c["weights"].double()
    dy = torch.zeros(c["dy"].shape, dtype=torch.float64, device="cuda")
    dw = torch.empty((T, k), dtype=torch.float64, device="cuda")
    dx = torch.empty((T, H), dtype=torch.float64, device="cuda")
    for t0 in range(0, T, 512):
        at = dest[t0: t0 + 512]
        d = c["dout"][t0: t0 + 512].double()
        dy[at.flatten()] = (w[t0: t0 + 512, :, None] * d[:, None]).flatten(0, 1)
        dw[t0: t0 + 512] = (c["y"][at].double() * d[:, None]).sum(-1)
        dx[t0: t0 + 512] = c["dxe"][at].double().sum(1)
    if c["residual"]:
        dx += c["dres"].double()
    # the softmax's Jacobian, row by row: diag(w) - w w^T
    ds = w * dw - w * (w * dw).sum(-1, keepdim=True)
    dlogits = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    dlogits[torch.arange(T, device="cuda")[:, None], c["ids"].long()] = ds
    got = {"dy": dy, "dweights": dw, "dlogits": dlogits, "dx": dx}
    if c["bias"]:
        got["dbias"] = dlogits.T @ torch.ones(T, dtype=torch.float64, device="cuda")
    return got


def exact(case, seed):
    c = prepare(case, seed)
    return {"linear": _exact_linear, "linear_grad": _exact_linear_grad, "swiglu_grad": _exact_swiglu_grad,
            "dispatch_grad": _exact_dispatch_grad}[c["op"]](c)
