"""The decode-side operators of moe_glue, case by case: RMS norm with the residual's addition (bf16, E4M3 with one
fp32 scale per column group, or MXFP8 out), products with MXFP4 weights for a few tokens, and the whole
Mixture-of-Experts layer for a few tokens (bf16 or MXFP4 expert weights).

A case is run in its plain form, in elementary torch operations in fp32, or (``own``) by the library's calls.  Codes
are returned as the float8 values that they stand for."""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # the norm before one decoded token's router, at the Qwen3-30B-A3B width: latency alone
        {"name": "norm one token", "op": "norm", "T": 1, "H": 2048, "fmt": "bf16", "group": 0, "residual": True,
         "normed": False},
        # the same norm over the benchmark's prefill batch
        {"name": "norm prefill", "op": "norm", "T": 4096, "H": 2048, "fmt": "bf16", "group": 0, "residual": True,
         "normed": False},
        # FP8 experts: codes and scales for the experts, the bf16 row for the router; an odd token count
        {"name": "norm fp8 odd", "op": "norm", "T": 1023, "H": 4096, "fmt": "fp8", "group": 128, "residual": True,
         "normed": True},
        # MXFP8 experts at the DeepSeek-V3 width and batch, the largest norm
        {"name": "norm mxfp8 large", "op": "norm", "T": 8192, "H": 7168, "fmt": "mxfp8", "group": 32,
         "residual": True, "normed": False},
        # a shared expert's gate and up rows at the DeepSeek-V3 shape, one token
        {"name": "linear one token", "op": "linear", "T": 1, "K": 7168, "N": 4096},
        # its down rows, an odd handful of tokens
        {"name": "linear odd", "op": "linear", "T": 13, "K": 2048, "N": 7168},
        # a wide dense projection at the largest batch the call takes
        {"name": "linear wide", "op": "linear", "T": 64, "K": 7168, "N": 16384},
        # the tiny workload as one layer call: launch latency
        {"name": "layer tiny", "op": "layer", "T": 16, "H": 256, "E": 8, "k": 2, "I": 128, "fmt": "bf16",
         "bias": False, "zipf": 0.0},
        # one user's decode step at the Qwen3-30B-A3B shape: k experts' weights
        {"name": "layer one token", "op": "layer", "T": 1, "H": 2048, "E": 128, "k": 8, "I": 768, "fmt": "bf16",
         "bias": False, "zipf": 0.0},
        # the decode workload: nearly every expert's weights once
        {"name": "layer decode", "op": "layer", "T": 32, "H": 2048, "E": 128, "k": 8, "I": 768, "fmt": "bf16",
         "bias": False, "zipf": 0.0},
        # 4-bit experts under skewed routing: some experts have most tokens, an odd batch near the limit
        {"name": "layer mxfp4 skewed", "op": "layer", "T": 61, "H": 4096, "E": 64, "k": 6, "I": 1408,
         "fmt": "mxfp4", "bias": False, "zipf": 1.2},
        # 4-bit experts at the DeepSeek-V3 shape with the router bias, the most bytes
        {"name": "layer mxfp4 large", "op": "layer", "T": 16, "H": 7168, "E": 256, "k": 8, "I": 2048,
         "fmt": "mxfp4", "bias": True, "zipf": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "linear", "layer", "layer", "layer"))
    if op == "norm":
        fmt = rng.choice(("bf16", "fp8", "mxfp8"))
        group = {"bf16": 0, "fp8": rng.choice((16, 32, 64, 128, 256)), "mxfp8": 32}[fmt]
        unit = max(8, group)
        T = _log(rng, 1, 8192)
        H = unit * _log(rng, 256 // unit, 8192 // unit)
        while T * H > 8192 * 7168:
            T = max(1, T // 2 + rng.randrange(2))
        return {"op": op, "T": T, "H": H, "fmt": fmt, "group": group, "residual": rng.random() < 0.7,
                "normed": fmt != "bf16" and rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 64), "K": 32 * _log(rng, 8, 224), "N": _log(rng, 64, 16384)}
    fmt = rng.choice(("bf16", "mxfp4"))
    unit = 8 if fmt == "bf16" else 32
    while True:
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 64)
        H = unit * _log(rng, 256 // unit, 7168 // unit)
        I = unit * _log(rng, 64 // unit, 2048 // unit)
        c = {"op": op, "T": T, "H": H, "E": E, "k": k, "I": I, "fmt": fmt, "bias": rng.random() < 0.3,
             "zipf": rng.choice((0.0, 0.0, 1.2))}
        if 6 * E * I * H <= 6 << 30 and T * k * I * H <= 32 * 8 * 768 * 2048 * 2:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, std, g):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _mxfp4(rows, g):
    """Random E2M1 codes, two to a byte, and E8M0 scale bytes; values of a trained layer's size, about 0.02."""
    *lead, K = rows
    codes = torch.randint(0, 256, (*lead, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 122, (*lead, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        c["x"] = _normal((T, H), 1.0, g)
        c["r"] = _normal((T, H), 4.0, g) if c["residual"] else None
        c["w"] = (1.0 + 0.2 * _normal((H,), 1.0, g).float()).to(torch.bfloat16)
        c["residual_out"] = torch.empty_like(c["x"]) if c["residual"] else None
        if c["fmt"] == "bf16" or c["normed"]:
            c["out"] = torch.empty_like(c["x"])
        else:
            c["out"] = None
        if c["fmt"] != "bf16":
            c["codes"] = torch.empty((T, H), dtype=torch.uint8, device="cuda")
            c["scales"] = torch.empty((T, H // c["group"]), device="cuda",
                                      dtype=torch.float32 if c["fmt"] == "fp8" else torch.uint8)
    elif c["op"] == "linear":
        c["x"] = _normal((c["T"], c["K"]), 1.0, g)
        c["codes"], c["scales"] = _mxfp4((c["N"], c["K"]), g)
        c["out"] = torch.empty((c["T"], c["N"]), dtype=torch.bfloat16, device="cuda")
    else:
        T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
        c["x"] = _normal((T, H), 1.0, g)
        logits = torch.empty((T, E), device="cuda").normal_(generator=g)
        if c["zipf"] > 0.0:
            rank = torch.randperm(E, device="cuda", generator=g) + 1
            logits = logits - c["zipf"] * torch.log(rank.float())
        c["logits"] = logits
        c["bias_t"] = torch.empty((E,), device="cuda").normal_(0.0, 0.5, generator=g) if c["bias"] else None
        if c["fmt"] == "bf16":
            c["wgu"], c["wd"] = _normal((E, 2 * I, H), 0.02, g), _normal((E, H, I), 0.02, g)
        else:
            c["wgu"], c["sgu"] = _mxfp4((E, 2 * I, H), g)
            c["wd"], c["sd"] = _mxfp4((E, H, I), g)
        c["bufs"] = {"topk_ids": torch.empty((T, k), dtype=torch.int32, device="cuda"),
                     "topk_weights": torch.empty((T, k), dtype=torch.float32, device="cuda"),
                     "out": torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
                     # the slots' activations between the layer's two products
                     "workspace": torch.empty((T * k * I * 4 + (1 << 16),), dtype=torch.uint8, device="cuda")}
    return c


# --------------------------------------------------------------- plain forms
def _plain_norm(c):
    s = c["x"].float()
    got = {}
    if c["residual"]:
        s = s + c["r"].float()
        got["residual_out"] = s.to(torch.bfloat16)
    n = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * c["w"].float()
    if c["fmt"] == "bf16" or c["normed"]:
        got["out"] = n.to(torch.bfloat16)
    if c["fmt"] != "bf16":
        b = n.reshape(c["T"], -1, c["group"])
        amax = b.abs().amax(-1, keepdim=True)
        if c["fmt"] == "fp8":
            inv = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
            got["scales"] = (amax / 448.0)[..., 0]
        else:
            # amax = m * 2^x with m in [1/2, 1): floor(log2 amax) = x - 1
            e = torch.where(amax > 0, (torch.frexp(amax).exponent - 9).clamp(min=-127), -127)
            inv = torch.ldexp(torch.ones_like(amax), -e)
            got["scales"] = (e + 127)[..., 0].to(torch.uint8).view(torch.float8_e8m0fnu)
        q = (b * inv).clamp(-448.0, 448.0)
        got["codes"] = q.reshape(c["T"], c["H"]).to(torch.float8_e4m3fn)
    return got


def _values(codes, scales):
    """The fp32 values of E2M1 codes (low nibble first) and E8M0 scales."""
    lut = torch.tensor(E2M1, device=codes.device)
    pair = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), -1)  # byte -> its two values
    v = pair[codes.int()].reshape(*codes.shape[:-1], -1, 32)
    s = torch.exp2(scales.float() - 127.0)
    return (v * s[..., None]).flatten(-2)


def _plain_linear(c):
    return (c["x"].float() @ _values(c["codes"], c["scales"]).T).to(torch.bfloat16)


def _plain_layer(c):
    key = c["logits"] if c["bias_t"] is None else c["logits"] + c["bias_t"]
    top, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    top, ids = top[:, : c["k"]], ids[:, : c["k"]]
    ex = torch.exp(top - top[:, :1])
    w = ex / ex.sum(-1, keepdim=True)
    e = ids.reshape(-1)
    if c["fmt"] == "bf16":
        wgu = c["wgu"][e].float()
    else:
        wgu = _values(c["wgu"][e], c["sgu"][e])
    x = c["x"].float().repeat_interleave(c["k"], 0)
    h = torch.bmm(wgu, x[:, :, None])[:, :, 0]
    del wgu
    gate, up = h[:, : c["I"]], h[:, c["I"]:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    if c["fmt"] == "bf16":
        wd = c["wd"][e].float()
    else:
        wd = _values(c["wd"][e], c["sd"][e])
    y = torch.bmm(wd, act[:, :, None])[:, :, 0].reshape(c["T"], c["k"], c["H"])
    out = (w[:, :, None] * y).sum(1).to(torch.bfloat16)
    return {"topk_ids": ids.int(), "topk_weights": w, "out": out}


# --------------------------------------------------------- the library's calls
def _own_norm(c):
    import moe_glue_amd as mg

    if c["fmt"] == "bf16":
        out, res = mg.rmsnorm(c["x"], c["w"], c["r"], eps=EPS, out=c["out"], residual_out=c["residual_out"])
        return {"out": out, "residual_out": res} if c["residual"] else {"out": out}
    if c["fmt"] == "fp8":
        codes, scales, res = mg.rmsnorm_fp8(c["x"], c["w"], c["group"], c["r"], eps=EPS, out=c["codes"],
                                            scales=c["scales"], residual_out=c["residual_out"], normed=c["out"])
    else:
        codes, scales, res = mg.rmsnorm_mxfp8(c["x"], c["w"], c["r"], eps=EPS, out=c["codes"], scales=c["scales"],
                                              residual_out=c["residual_out"], normed=c["out"])
        scales = scales.view(torch.float8_e8m0fnu)
    got = {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if c["residual"]:
        got["residual_out"] = res
    if c["normed"]:
        got["out"] = c["out"]
    return got


def _own_layer(c):
    import moe_glue_amd as mg

    if c["fmt"] == "bf16":
        r = mg.decode_layer(c["logits"], c["k"], c["x"], c["wgu"], c["wd"], bias=c["bias_t"], out=c["bufs"])
    else:
        r = mg.decode_layer_mxfp4(c["logits"], c["k"], c["x"], c["wgu"], c["sgu"], c["wd"], c["sd"],
                                  bias=c["bias_t"], out=c["bufs"])
    return {"topk_ids": r["topk_ids"], "topk_weights": r["topk_weights"], "out": r["out"]}


def run(state):
    op = state["op"]
    if own:
        if op == "norm":
            return _own_norm(state)
        if op == "linear":
            import moe_glue_amd as mg

            return mg.linear_mxfp4(state["x"], state["codes"], state["scales"], out=state["out"])
        return _own_layer(state)
    return {"norm": _plain_norm, "linear": _plain_linear, "layer": _plain_layer}[op](state)


# --------------------------------------------------------------------- work
def _active_experts(c):
    """Distinct experts a batch picks, the mean of a few simulated ones of the case's distribution."""
    rng = np.random.default_rng(1)
    n = 0
    for _ in range(4):
        z = rng.standard_normal((c["T"], c["E"]))
        if c["bias"]:
            z = z + 0.5 * rng.standard_normal(c["E"])
        if c["zipf"] > 0.0:
            z = z - c["zipf"] * np.log(np.arange(1, c["E"] + 1))
        n += np.unique(np.argsort(-z, axis=1)[:, : c["k"]]).size
    return n / 4


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        b = 2 * H + T * H * (2 + (4 if case["residual"] else 0))
        if case["fmt"] == "bf16":
            b += 2 * T * H
        else:
            b += T * H + T * (H // case["group"]) * (4 if case["fmt"] == "fp8" else 1)
            b += 2 * T * H if case["normed"] else 0
        return {"bytes": b, "flops": 6 * T * H}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": N * K / 2 + N * K / 32 + 2 * T * (K + N), "flops": 2 * T * K * N}
    T, H, E, k, I = case["T"], case["H"], case["E"], case["k"], case["I"]
    per = 2.0 if case["fmt"] == "bf16" else 0.5 + 1 / 32
    return {"bytes": _active_experts(case) * 3 * I * H * per + 4 * T * E + 8 * T * k + 4 * T * H,
            "flops": 6 * T * k * I * H}


# ------------------------------------------------------------- 64-bit values
def _e2m1_f64(codes, scales):
    """Values from the format's fields: sign, 2 exponent bits of bias 1, 1 mantissa bit; subnormal below 1."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign = torch.where(nib >= 8, -1.0, 1.0)
    mag = nib - 8.0 * (nib >= 8)
    ex, m = torch.floor(mag / 2), mag % 2
    v = sign * torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (ex - 1))
    return v * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)


def _e4m3_f64(q):
    """q rounded to E4M3 (3 mantissa bits, least exponent -6, ties to even), saturating at 448."""
    q = q.clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    e = e - (2.0 ** e > q.abs()).double() * (e > -6) + (2.0 ** (e + 1) <= q.abs()).double()
    step = 2.0 ** (e - 3)
    return torch.round(q / step) * step


def _exact_norm(c):
    s = c["x"].double()
    got = {}
    if c["residual"]:
        s = s + c["r"].double()
        got["residual_out"] = s
    n = c["w"].double() * s / torch.sqrt(torch.linalg.vector_norm(s, dim=-1, keepdim=True) ** 2 / c["H"] + EPS)
    if c["fmt"] == "bf16" or c["normed"]:
        got["out"] = n
    if c["fmt"] != "bf16":
        b = n.unflatten(-1, (-1, c["group"]))
        amax = torch.maximum(b.max(-1).values, -b.min(-1).values)
        if c["fmt"] == "fp8":
            scale = amax / 448
        else:
            x = torch.floor(torch.log2(amax))
            x = x - (2.0 ** x > amax).double() + (2.0 ** (x + 1) <= amax).double()
            scale = 2.0 ** (x - 8)
        got["scales"] = scale
        got["codes"] = _e4m3_f64(b / scale[..., None]).flatten(-2)
    return got


def _exact_layer(c):
    key = c["logits"] if c["bias_t"] is None else c["logits"] + c["bias_t"]  # the keys are fp32 by definition
    top, ids = torch.topk(key.double(), c["k"])
    w = torch.softmax(top, -1)
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if c["fmt"] == "bf16":
            wgu, wd = c["wgu"][e].double(), c["wd"][e].double()
        else:
            wgu, wd = _e2m1_f64(c["wgu"][e], c["sgu"][e]), _e2m1_f64(c["wd"][e], c["sd"][e])
        gate, up = (c["x"][t].double() @ wgu.T).chunk(2, -1)
        out.index_add_(0, t, w[t, j][:, None] * ((gate * torch.sigmoid(gate) * up) @ wd.T))
    return {"topk_ids": None, "topk_weights": w, "out": out}


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        return _exact_norm(c)
    if c["op"] == "linear":
        return torch.cat([c["x"].double() @ _e2m1_f64(q, s).T
                          for q, s in zip(c["codes"].split(1024), c["scales"].split(1024))], 1)
    return _exact_layer(c)
