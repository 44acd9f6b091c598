"""moe_glue_amd: the memory-bound Mixture-of-Experts glue path on MI355X (gfx950).

Four calls, each a thin wrapper over the C ABI of the HIP library
(include/moe_glue.h):

    route(logits, k, bias=None)        softmax top-k, expert counts/offsets,
                                       permutation maps
    expand_rows(x, dest_of_src, k)     expandInputRows: token rows -> expert rows
    swiglu(h)                          doActivation: silu(gate) * up
    combine(y, topk_weights, dest_of_src)  weighted sum back to token order
    route_expand(logits, k, x, bias=None)  route + expand, one launch for T <= 64
    route_expand_noalloc(logits, k, x, out=...)  the same with the library's built-in
                                       workspace (allocates nothing given `out`)
    route_padded(logits, k, pad_to)    route with expert segments padded to pad_to rows
    expand_rows_fp8(x, dest, k, group) expand with FP8 E4M3 quantisation per column group
    expand_rows_mxfp8(x, dest, k)    expand with MXFP8 quantisation (E8M0 scale per 32 columns)
    route_expand_fp8 / route_expand_mxfp8  route + the quantising expand in one call
    rmsnorm(x, weight, residual)       root-mean-square norm with the residual's addition
    rmsnorm_fp8 / rmsnorm_mxfp8        the same with E4M3 codes and fp32 or E8M0 scales out
    decode_layer(logits, k, x, w_gate_up, w_down)  the whole layer for T <= 64 tokens, experts included
    decode_layer_mxfp4(...)            the same on 4-bit (MXFP4) expert weights
    linear_mxfp4(x, w, scales)         product of T <= 64 tokens with MXFP4 weights

Tensors are torch CUDA (HIP) tensors; bf16 tensors use torch.bfloat16.  Work
is enqueued on torch's current stream and nothing synchronises.  Every call
accepts preallocated outputs (``out=`` / the route output dict) so a caller
can run the path without allocating.
"""
from __future__ import annotations

from ._binding import (DECODE_T_MAX, E_MAX, EXPORTED, K_MAX, LIB_PATH, NORM_H_MAX,  # noqa: F401
                       MoEGlueArgumentError, MoEGlueError, check, load)

__all__ = ["route", "route_workspace_bytes", "alloc_route_outputs", "route_padded", "padded_rows", "expand_rows",
           "expand_rows_fp8", "expand_rows_mxfp8",
           "route_expand", "route_expand_noalloc", "noalloc_scratch_bytes", "route_expand_padded", "route_expand_fp8", "route_expand_mxfp8", "swiglu", "combine",
           "rmsnorm", "rmsnorm_fp8", "rmsnorm_mxfp8", "decode_layer", "decode_layer_mxfp4",
           "decode_layer_workspace_bytes", "alloc_decode_outputs", "linear_mxfp4",
           "copy_probe", "mix_probe", "MoEGlueError", "MoEGlueArgumentError", "E_MAX", "K_MAX",
           "NORM_H_MAX", "DECODE_T_MAX"]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


_raw_stream = None


def _stream(device) -> int:
    """Handle of torch's current stream on `device`."""
    global _raw_stream
    if _raw_stream is None:
        # torch's own getter of the handle makes no stream object on the way (0.12 us
        # a call, 1.87 with one), but torch does not promise it: without it the
        # documented one
        torch = _torch()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(device.index)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need_gpu(name: str, t, dtype=None, ndim=None) -> None:
    if t is None:
        raise MoEGlueArgumentError(1, f"{name} is required")
    if not t.is_cuda:
        raise MoEGlueArgumentError(2, f"{name} must be a GPU tensor (got device {t.device})")
    if not t.is_contiguous():
        raise MoEGlueArgumentError(2, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise MoEGlueArgumentError(2, f"{name} must be {dtype} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise MoEGlueArgumentError(2, f"{name} must have {ndim} dims (got shape {tuple(t.shape)})")


def _check_bias(bias, E: int) -> None:
    """bias: None, or fp32 [E] on the GPU (the kernels read bias[e] for every e < E)."""
    if bias is None:
        return
    torch = _torch()
    _need_gpu("bias", bias, torch.float32, 1)
    if bias.shape[0] != E:
        raise MoEGlueArgumentError(2, f"bias has {bias.shape[0]} entries, logits has E={E}")


def _check_vec(name: str, t, dtype, n: int, at_least: bool = False) -> None:
    """t: a GPU tensor of `dtype` with exactly n (or at least n) elements."""
    _need_gpu(name, t, dtype)
    if (t.numel() < n) if at_least else (t.numel() != n):
        raise MoEGlueArgumentError(2, f"{name} has {t.numel()} entries, expected {'at least ' if at_least else ''}{n}")


def _check_route_out(out: dict, T: int, E: int, k: int, rows: int) -> None:
    """Caller-supplied route outputs: ids/weights/dest_of_src [T*k], offsets
    [E+1], counts [E] (or absent), src_of_dest at least `rows` entries (the
    padded row bound for a padded layout).  The workspace size is checked by
    the library itself, which receives its byte count."""
    torch = _torch()
    _check_vec("topk_ids", out.get("topk_ids"), torch.int32, T * k)
    _check_vec("topk_weights", out.get("topk_weights"), torch.float32, T * k)
    _check_vec("expert_offsets", out.get("expert_offsets"), torch.int32, E + 1)
    if out.get("expert_counts") is not None:
        _check_vec("expert_counts", out["expert_counts"], torch.int32, E)
    _check_vec("dest_of_src", out.get("dest_of_src"), torch.int32, T * k)
    _check_vec("src_of_dest", out.get("src_of_dest"), torch.int32, rows, at_least=True)
    ws = out.get("workspace")
    if ws is not None:
        _need_gpu("workspace", ws)


def _check_rows_out(name: str, t, rows: int, width: int, dtype) -> None:
    """t: a 2-D GPU tensor of `dtype`, [>= rows, width]."""
    _need_gpu(name, t, dtype, 2)
    if t.shape[0] < rows or t.shape[1] != width:
        raise MoEGlueArgumentError(2, f"{name} is {list(t.shape)}, expected [>= {rows}, {width}]")


def route_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(load().moe_route_workspace_bytes(T, E, k))


def alloc_route_outputs(T: int, E: int, k: int, device) -> dict:
    """Device buffers for route(): ids, weights, offsets, counts, maps, workspace."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    return {
        "topk_ids": torch.empty((T, k), dtype=i32, device=device),
        "topk_weights": torch.empty((T, k), dtype=f32, device=device),
        "expert_offsets": torch.empty((E + 1,), dtype=i32, device=device),
        "expert_counts": torch.empty((E,), dtype=i32, device=device),
        "dest_of_src": torch.empty((T * k,), dtype=i32, device=device),
        "src_of_dest": torch.empty((T * k,), dtype=i32, device=device),
        "workspace": torch.empty((max(16, route_workspace_bytes(T, E, k)),), dtype=torch.uint8, device=device),
    }


def route(logits, k: int, bias=None, out: dict | None = None) -> dict:
    """Softmax top-k routing and dispatch bookkeeping; see moe_route in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    T, E = logits.shape
    _check_bias(bias, E)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
    _check_route_out(out, T, E, k, T * k)
    ws = out["workspace"]
    lib = load()
    st = lib.moe_route(_ptr(logits), _ptr(bias), T, E, k, _ptr(out["topk_ids"]), _ptr(out["topk_weights"]),
                       _ptr(out["expert_offsets"]), _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]),
                       _ptr(out["src_of_dest"]), _ptr(ws), ws.numel() if ws is not None else 0,
                       _stream(logits.device))
    check(st, "moe_route")
    return out


def padded_rows(T: int, E: int, k: int, pad_to: int) -> int:
    """Upper bound on the rows of the padded layout: T*k + E*(pad_to-1)."""
    return int(load().moe_route_padded_rows(T, E, k, pad_to))


def route_padded(logits, k: int, pad_to: int, bias=None, out: dict | None = None) -> dict:
    """route() with each expert's segment padded to a multiple of pad_to rows;
    src_of_dest has padded_rows() entries (-1 on padding rows, valid up to
    expert_offsets[E]).  See moe_route_padded in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    T, E = logits.shape
    _check_bias(bias, E)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
        out["src_of_dest"] = torch.empty((max(1, padded_rows(T, E, k, pad_to)),), dtype=torch.int32,
                                         device=logits.device)
    _check_route_out(out, T, E, k, padded_rows(T, E, k, pad_to))
    ws = out["workspace"]
    st = load().moe_route_padded(_ptr(logits), _ptr(bias), T, E, k, pad_to, _ptr(out["topk_ids"]),
                                 _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                 _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]), _ptr(out["src_of_dest"]),
                                 _ptr(ws), ws.numel() if ws is not None else 0, _stream(logits.device))
    check(st, "moe_route_padded")
    return out


def route_expand_padded(logits, k: int, pad_to: int, x, bias=None, out: dict | None = None) -> dict:
    """route_padded() and expand_rows() in one call; see moe_route_expand_padded
    in include/moe_glue.h.  x_expanded has padded_rows() rows (padding rows
    are not written)."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    H = x.shape[1]
    _check_bias(bias, E)
    P = max(1, padded_rows(T, E, k, pad_to))
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
        out["src_of_dest"] = torch.empty((P,), dtype=torch.int32, device=logits.device)
    if out.get("x_expanded") is None:
        out["x_expanded"] = torch.empty((P, H), dtype=torch.bfloat16, device=x.device)
    _check_route_out(out, T, E, k, padded_rows(T, E, k, pad_to))
    _check_rows_out("x_expanded", out["x_expanded"], padded_rows(T, E, k, pad_to), H, torch.bfloat16)
    ws = out["workspace"]
    st = load().moe_route_expand_padded(_ptr(logits), _ptr(bias), T, E, k, pad_to, _ptr(x), H, _ptr(out["topk_ids"]),
                                        _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                        _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]),
                                        _ptr(out["src_of_dest"]), _ptr(out["x_expanded"]), _ptr(ws),
                                        ws.numel() if ws is not None else 0, _stream(logits.device))
    check(st, "moe_route_expand_padded")
    return out


def route_expand_fp8(logits, k: int, x, group: int, pad_to: int = 1, bias=None, out: dict | None = None) -> dict:
    """route_padded() (route() for pad_to = 1) and expand_rows_fp8() in one
    call; see moe_route_expand_fp8 in include/moe_glue.h.  Returns the route
    dict plus "x_expanded" (uint8 E4M3 codes [rows, H]) and "scales" (fp32
    [rows, H/group]); padding rows are not written."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    H = x.shape[1]
    _check_bias(bias, E)
    P = max(1, padded_rows(T, E, k, pad_to)) if pad_to > 1 else max(1, T * k)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
        out["src_of_dest"] = torch.empty((P,), dtype=torch.int32, device=logits.device)
    if out.get("x_expanded") is None:
        out["x_expanded"] = torch.empty((P, H), dtype=torch.uint8, device=x.device)
    if out.get("scales") is None:
        out["scales"] = torch.empty((P, max(1, H // group)), dtype=torch.float32, device=x.device)
    rows = padded_rows(T, E, k, pad_to) if pad_to > 1 else T * k
    _check_route_out(out, T, E, k, rows)
    _check_rows_out("x_expanded", out["x_expanded"], rows, H, torch.uint8)
    _check_rows_out("scales", out["scales"], rows, H // group if group > 0 and H % group == 0 else -1,
                    torch.float32)
    ws = out["workspace"]
    st = load().moe_route_expand_fp8(_ptr(logits), _ptr(bias), T, E, k, pad_to, _ptr(x), H, group,
                                     _ptr(out["topk_ids"]), _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                     _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]),
                                     _ptr(out["src_of_dest"]), _ptr(out["x_expanded"]), _ptr(out["scales"]),
                                     _ptr(ws), ws.numel() if ws is not None else 0, _stream(logits.device))
    check(st, "moe_route_expand_fp8")
    return out


def route_expand_mxfp8(logits, k: int, x, pad_to: int = 1, bias=None, out: dict | None = None) -> dict:
    """route_padded() (route() for pad_to = 1) and expand_rows_mxfp8() in one
    call; see moe_route_expand_mxfp8 in include/moe_glue.h.  Returns the route
    dict plus "x_expanded" (uint8 E4M3 codes [rows, H]) and "scales" (uint8
    E8M0 bytes [rows, H/32]); padding rows are not written."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    H = x.shape[1]
    _check_bias(bias, E)
    P = max(1, padded_rows(T, E, k, pad_to)) if pad_to > 1 else max(1, T * k)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
        out["src_of_dest"] = torch.empty((P,), dtype=torch.int32, device=logits.device)
    if out.get("x_expanded") is None:
        out["x_expanded"] = torch.empty((P, H), dtype=torch.uint8, device=x.device)
    if out.get("scales") is None:
        out["scales"] = torch.empty((P, max(1, H // 32)), dtype=torch.uint8, device=x.device)
    rows = padded_rows(T, E, k, pad_to) if pad_to > 1 else T * k
    _check_route_out(out, T, E, k, rows)
    _check_rows_out("x_expanded", out["x_expanded"], rows, H, torch.uint8)
    _check_rows_out("scales", out["scales"], rows, H // 32 if H % 32 == 0 else -1, torch.uint8)
    ws = out["workspace"]
    st = load().moe_route_expand_mxfp8(_ptr(logits), _ptr(bias), T, E, k, pad_to, _ptr(x), H,
                                       _ptr(out["topk_ids"]), _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                       _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]),
                                       _ptr(out["src_of_dest"]), _ptr(out["x_expanded"]), _ptr(out["scales"]),
                                       _ptr(ws), ws.numel() if ws is not None else 0, _stream(logits.device))
    check(st, "moe_route_expand_mxfp8")
    return out


def expand_rows(x, dest_of_src, k: int, out=None):
    """x_expanded[dest_of_src[t*k+j]] = x[t]; see moe_expand_rows in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("x", x, torch.bfloat16, 2)
    _need_gpu("dest_of_src", dest_of_src, torch.int32)
    T, H = x.shape
    if dest_of_src.numel() != T * k:
        raise MoEGlueArgumentError(2, f"dest_of_src has {dest_of_src.numel()} entries, expected T*k={T * k}")
    if out is None:
        out = torch.empty((T * k, H), dtype=torch.bfloat16, device=x.device)
    else:
        _need_gpu("out", out, torch.bfloat16, 2)
        if out.shape[0] < T * k or out.shape[1] != H:
            raise MoEGlueArgumentError(2, f"out must be [>= {T * k}, {H}] (more rows for a padded layout)")
    st = load().moe_expand_rows(_ptr(x), _ptr(dest_of_src), T, H, k, _ptr(out), _stream(x.device))
    check(st, "moe_expand_rows")
    return out


def expand_rows_fp8(x, dest_of_src, k: int, group: int, rows: int | None = None, out=None, scales=None):
    """FP8 (E4M3) quantising expand; returns (codes uint8 [rows, H], scales fp32
    [rows, H/group]).  See moe_expand_rows_fp8 in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("x", x, torch.bfloat16, 2)
    _need_gpu("dest_of_src", dest_of_src, torch.int32)
    T, H = x.shape
    if dest_of_src.numel() != T * k:
        raise MoEGlueArgumentError(2, f"dest_of_src has {dest_of_src.numel()} entries, expected T*k={T * k}")
    n = T * k if rows is None else rows
    if n < T * k:
        raise MoEGlueArgumentError(2, f"rows={n} is below T*k={T * k}")
    if out is None:
        out = torch.empty((n, H), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, max(1, H // group)), dtype=torch.float32, device=x.device)
    _check_rows_out("out", out, n, H, torch.uint8)
    _check_rows_out("scales", scales, n, H // group if group > 0 and H % group == 0 else -1, torch.float32)
    st = load().moe_expand_rows_fp8(_ptr(x), _ptr(dest_of_src), T, H, k, group, _ptr(out), _ptr(scales),
                                    _stream(x.device))
    check(st, "moe_expand_rows_fp8")
    return out, scales


def expand_rows_mxfp8(x, dest_of_src, k: int, rows: int | None = None, out=None, scales=None):
    """MXFP8 quantising expand; returns (codes uint8 [rows, H], E8M0 scale bytes
    uint8 [rows, H/32]).  See moe_expand_rows_mxfp8 in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("x", x, torch.bfloat16, 2)
    _need_gpu("dest_of_src", dest_of_src, torch.int32)
    T, H = x.shape
    if dest_of_src.numel() != T * k:
        raise MoEGlueArgumentError(2, f"dest_of_src has {dest_of_src.numel()} entries, expected T*k={T * k}")
    n = T * k if rows is None else rows
    if n < T * k:
        raise MoEGlueArgumentError(2, f"rows={n} is below T*k={T * k}")
    if out is None:
        out = torch.empty((n, H), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((n, max(1, H // 32)), dtype=torch.uint8, device=x.device)
    _check_rows_out("out", out, n, H, torch.uint8)
    _check_rows_out("scales", scales, n, H // 32 if H % 32 == 0 else -1, torch.uint8)
    st = load().moe_expand_rows_mxfp8(_ptr(x), _ptr(dest_of_src), T, H, k, _ptr(out), _ptr(scales),
                                      _stream(x.device))
    check(st, "moe_expand_rows_mxfp8")
    return out, scales


def route_expand(logits, k: int, x, bias=None, out: dict | None = None) -> dict:
    """route() and expand_rows() in one call (one launch for T <= 64); see
    moe_route_expand in include/moe_glue.h.  Returns route()'s dict plus
    "x_expanded"."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    H = x.shape[1]
    _check_bias(bias, E)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
    if out.get("x_expanded") is None:
        out["x_expanded"] = torch.empty((T * k, H), dtype=torch.bfloat16, device=x.device)
    _check_route_out(out, T, E, k, T * k)
    _check_rows_out("x_expanded", out["x_expanded"], T * k, H, torch.bfloat16)
    ws = out["workspace"]
    st = load().moe_route_expand(_ptr(logits), _ptr(bias), T, E, k, _ptr(x), H, _ptr(out["topk_ids"]),
                                 _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                 _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]), _ptr(out["src_of_dest"]),
                                 _ptr(out["x_expanded"]), _ptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(logits.device))
    check(st, "moe_route_expand")
    return out


def noalloc_scratch_bytes() -> int:
    """Bytes of the library's built-in scratch behind route_expand_noalloc()."""
    return int(load().moe_noalloc_scratch_bytes())


def route_expand_noalloc(logits, k: int, x, bias=None, out: dict | None = None) -> dict:
    """route_expand() with the library's built-in device scratch as the route
    workspace; see moe_route_expand_noalloc in include/moe_glue.h.  With `out`
    (the route dict without "workspace", plus "x_expanded") nothing is
    allocated.  Calls that can overlap on one GPU share the scratch and race."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    H = x.shape[1]
    _check_bias(bias, E)
    if out is None:
        out = alloc_route_outputs(T, E, k, logits.device)
        del out["workspace"]
        out["x_expanded"] = torch.empty((T * k, H), dtype=torch.bfloat16, device=x.device)
    _check_route_out(out, T, E, k, T * k)
    _check_rows_out("x_expanded", out.get("x_expanded"), T * k, H, torch.bfloat16)
    st = load().moe_route_expand_noalloc(_ptr(logits), _ptr(bias), T, E, k, _ptr(x), H, _ptr(out["topk_ids"]),
                                         _ptr(out["topk_weights"]), _ptr(out["expert_offsets"]),
                                         _ptr(out.get("expert_counts")), _ptr(out["dest_of_src"]),
                                         _ptr(out["src_of_dest"]), _ptr(out["x_expanded"]), _stream(logits.device))
    check(st, "moe_route_expand_noalloc")
    return out


def swiglu(h, out=None):
    """act = silu(h[:, :I]) * h[:, I:]; see moe_swiglu in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("h", h, torch.bfloat16, 2)
    R, I2 = h.shape
    if I2 % 2:
        raise MoEGlueArgumentError(2, f"h has an odd width {I2}; expected [R, 2I]")
    I = I2 // 2
    if out is None:
        out = torch.empty((R, I), dtype=torch.bfloat16, device=h.device)
    else:
        _need_gpu("out", out, torch.bfloat16, 2)
        if tuple(out.shape) != (R, I):
            raise MoEGlueArgumentError(2, f"out must be [{R}, {I}]")
    st = load().moe_swiglu(_ptr(h), R, I, _ptr(out), _stream(h.device))
    check(st, "moe_swiglu")
    return out


def combine(y, topk_weights, dest_of_src, out=None):
    """out[t] = sum_j w[t,j] * y[dest_of_src[t*k+j]]; see moe_combine in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("y", y, torch.bfloat16, 2)
    _need_gpu("topk_weights", topk_weights, torch.float32, 2)
    _need_gpu("dest_of_src", dest_of_src, torch.int32)
    T, k = topk_weights.shape
    R, H = y.shape
    if R < T * k or dest_of_src.numel() != T * k:
        raise MoEGlueArgumentError(2, f"y has {R} rows and dest_of_src {dest_of_src.numel()}; expected T*k={T * k} "
                                      "entries and at least as many rows")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    else:
        _need_gpu("out", out, torch.bfloat16, 2)
        if tuple(out.shape) != (T, H):
            raise MoEGlueArgumentError(2, f"out must be [{T}, {H}]")
    st = load().moe_combine(_ptr(y), _ptr(topk_weights), _ptr(dest_of_src), T, H, k, _ptr(out), _stream(y.device))
    check(st, "moe_combine")
    return out


def _same_device(named, device) -> None:
    """Every given tensor lives on `device` (a kernel runs on one GPU)."""
    for name, t in named:
        if t is not None and t.device != device:
            raise MoEGlueArgumentError(2, f"{name} is on {t.device}, expected {device}")


def _check_shape(name: str, t, dtype, shape: tuple, device) -> None:
    """t: a contiguous GPU tensor of this dtype and shape on `device`."""
    if t is not None and t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    _need_gpu(name, t, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise MoEGlueArgumentError(2, f"{name} is {list(t.shape)}, expected {list(shape)}")
    _same_device([(name, t)], device)


def _enqueue(fn: str, device, *args) -> None:
    """Call the library on `device`'s current stream, with `device` current (the
    default stream's handle names no device of its own)."""
    torch = _torch()
    call = getattr(load(), fn)
    if torch.cuda.current_device() == device.index:
        status = call(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = call(*args, _stream(device))
    if status:
        check(status, fn)


def _norm_args(x, weight, residual, residual_out, out, normed_name: str):
    """Checks shared by the norms; returns (T, H, residual_out)."""
    torch = _torch()
    bf16 = torch.bfloat16
    _need_gpu("x", x, bf16, 2)
    shape, dev = x.shape, x.device
    _check_shape("weight", weight, bf16, (shape[1],), dev)
    if residual is not None:
        _check_shape("residual", residual, bf16, shape, dev)
        if residual_out is None:
            residual_out = torch.empty_like(x)
        else:
            _check_shape("residual_out", residual_out, bf16, shape, dev)
    elif residual_out is not None:
        raise MoEGlueArgumentError(1, "residual_out without residual")
    if out is not None:
        _check_shape(normed_name, out, bf16, shape, dev)
    return shape[0], shape[1], residual_out


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, out=None, residual_out=None):
    """Root-mean-square norm of x (+ residual); returns (out, residual_out), the
    latter None without a residual.  residual_out may be `residual` itself.  See
    moe_rmsnorm in include/moe_glue.h."""
    T, H, residual_out = _norm_args(x, weight, residual, residual_out, out, "out")
    if out is None:
        out = _torch().empty_like(x)
    _enqueue("moe_rmsnorm", x.device, _ptr(x), _ptr(residual), _ptr(weight), T, H, eps, _ptr(residual_out), _ptr(out))
    return out, residual_out


def rmsnorm_fp8(x, weight, group: int, residual=None, eps: float = 1e-6, out=None, scales=None, residual_out=None,
                normed=None):
    """rmsnorm() with E4M3 codes and one fp32 scale per `group` columns; returns
    (codes uint8 [T, H], scales fp32 [T, H/group], residual_out).  `normed`: a
    bf16 [T, H] tensor that receives rmsnorm()'s row as well.  See
    moe_rmsnorm_fp8 in include/moe_glue.h."""
    torch = _torch()
    T, H, residual_out = _norm_args(x, weight, residual, residual_out, normed, "normed")
    if group < 1 or H % group != 0:
        raise MoEGlueArgumentError(2, f"group={group} does not divide H={H}")
    if out is None:
        out = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    else:
        _check_shape("out", out, torch.uint8, (T, H), x.device)
    if scales is None:
        scales = torch.empty((T, H // group), dtype=torch.float32, device=x.device)
    else:
        _check_shape("scales", scales, torch.float32, (T, H // group), x.device)
    _enqueue("moe_rmsnorm_fp8", x.device, _ptr(x), _ptr(residual), _ptr(weight), T, H, eps, group,
             _ptr(residual_out), _ptr(normed), _ptr(out), _ptr(scales))
    return out, scales, residual_out


def rmsnorm_mxfp8(x, weight, residual=None, eps: float = 1e-6, out=None, scales=None, residual_out=None, normed=None):
    """rmsnorm() with MXFP8 output; returns (codes uint8 [T, H], E8M0 scale bytes
    uint8 [T, H/32], residual_out).  `normed` as in rmsnorm_fp8().  See
    moe_rmsnorm_mxfp8 in include/moe_glue.h."""
    torch = _torch()
    T, H, residual_out = _norm_args(x, weight, residual, residual_out, normed, "normed")
    if H % 32 != 0:
        raise MoEGlueArgumentError(2, f"H={H} is not a multiple of the 32-column block")
    if out is None:
        out = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    else:
        _check_shape("out", out, torch.uint8, (T, H), x.device)
    if scales is None:
        scales = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    else:
        _check_shape("scales", scales, torch.uint8, (T, H // 32), x.device)
    _enqueue("moe_rmsnorm_mxfp8", x.device, _ptr(x), _ptr(residual), _ptr(weight), T, H, eps, _ptr(residual_out),
             _ptr(normed), _ptr(out), _ptr(scales))
    return out, scales, residual_out


def decode_layer_workspace_bytes(T: int, E: int, k: int, I: int) -> int:
    return int(load().moe_decode_layer_workspace_bytes(T, E, k, I))


def alloc_decode_outputs(T: int, E: int, k: int, H: int, I: int, device) -> dict:
    """Device buffers for decode_layer() and decode_layer_mxfp4(): ids, weights, out, workspace."""
    torch = _torch()
    return {
        "topk_ids": torch.empty((T, k), dtype=torch.int32, device=device),
        "topk_weights": torch.empty((T, k), dtype=torch.float32, device=device),
        "out": torch.empty((T, H), dtype=torch.bfloat16, device=device),
        "workspace": torch.empty((max(16, decode_layer_workspace_bytes(T, E, k, I)),), dtype=torch.uint8,
                                 device=device),
    }


def _decode_args(logits, k: int, x, w_gate_up, w_down, bias, out, mx: bool):
    """Checks shared by the two layers; returns (T, E, H, I, out)."""
    torch = _torch()
    _need_gpu("logits", logits, torch.float32, 2)
    _need_gpu("x", x, torch.bfloat16, 2)
    T, E = logits.shape
    H = x.shape[1]
    dev = x.device
    if x.shape[0] != T:
        raise MoEGlueArgumentError(2, f"x has {x.shape[0]} rows, logits has T={T}")
    if logits.device != dev or (bias is not None and bias.device != dev):
        _same_device([("logits", logits), ("bias", bias)], dev)
    _check_bias(bias, E)
    if w_gate_up is None or w_gate_up.dim() != 3:
        _need_gpu("w_gate_up", w_gate_up, None, 3)
    I = w_gate_up.shape[1] // 2
    if mx:
        if H % 32 != 0 or I % 32 != 0:
            raise MoEGlueArgumentError(2, f"H={H} and I={I} must be multiples of the 32-column block")
        _check_shape("w_gate_up", w_gate_up, torch.uint8, (E, 2 * I, H // 2), dev)
        _check_shape("w_down", w_down, torch.uint8, (E, H, I // 2), dev)
    else:
        _check_shape("w_gate_up", w_gate_up, torch.bfloat16, (E, 2 * I, H), dev)
        _check_shape("w_down", w_down, torch.bfloat16, (E, H, I), dev)
    if out is None:
        if not 0 < k <= min(E, K_MAX):
            raise MoEGlueArgumentError(2, f"k={k} must be in [1, {min(E, K_MAX)}]")
        out = alloc_decode_outputs(T, E, k, H, I, dev)
    else:
        _check_shape("topk_ids", out.get("topk_ids"), torch.int32, (T, k), dev)
        _check_shape("topk_weights", out.get("topk_weights"), torch.float32, (T, k), dev)
        _check_shape("out", out.get("out"), torch.bfloat16, (T, H), dev)
        ws = out.get("workspace")
        if ws is None or ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
            _need_gpu("workspace", ws, torch.uint8)
            _same_device([("workspace", ws)], dev)
    return T, E, H, I, out


def decode_layer(logits, k: int, x, w_gate_up, w_down, bias=None, out: dict | None = None) -> dict:
    """The whole layer for T <= DECODE_T_MAX tokens, routing and experts, in two
    launches: x [T, H], w_gate_up bf16 [E, 2I, H] (gate rows, then up rows),
    w_down bf16 [E, H, I].  Returns "topk_ids", "topk_weights", "out" [T, H] and
    the workspace.  See moe_decode_layer in include/moe_glue.h."""
    T, E, H, I, out = _decode_args(logits, k, x, w_gate_up, w_down, bias, out, False)
    ws = out["workspace"]
    _enqueue("moe_decode_layer", x.device, logits.data_ptr(), _ptr(bias), T, E, k, x.data_ptr(), H,
             w_gate_up.data_ptr(), w_down.data_ptr(), I, out["topk_ids"].data_ptr(), out["topk_weights"].data_ptr(),
             out["out"].data_ptr(), ws.data_ptr(), ws.numel())
    return out


def decode_layer_mxfp4(logits, k: int, x, w_gate_up, s_gate_up, w_down, s_down, bias=None,
                       out: dict | None = None) -> dict:
    """decode_layer() on MXFP4 expert weights: codes uint8 [E, 2I, H/2] and
    [E, H, I/2] (lower column in the low four bits), E8M0 scale bytes uint8
    [E, 2I, H/32] and [E, H, I/32].  See moe_decode_layer_mxfp4 in
    include/moe_glue.h."""
    u8 = _torch().uint8
    T, E, H, I, out = _decode_args(logits, k, x, w_gate_up, w_down, bias, out, True)
    _check_shape("s_gate_up", s_gate_up, u8, (E, 2 * I, H // 32), x.device)
    _check_shape("s_down", s_down, u8, (E, H, I // 32), x.device)
    ws = out["workspace"]
    _enqueue("moe_decode_layer_mxfp4", x.device, logits.data_ptr(), _ptr(bias), T, E, k, x.data_ptr(), H,
             w_gate_up.data_ptr(), s_gate_up.data_ptr(), w_down.data_ptr(), s_down.data_ptr(), I,
             out["topk_ids"].data_ptr(), out["topk_weights"].data_ptr(), out["out"].data_ptr(), ws.data_ptr(),
             ws.numel())
    return out


def linear_mxfp4(x, w, scales, out=None):
    """y = x W^T for T <= DECODE_T_MAX tokens and MXFP4 weights: codes uint8
    [N, K/2], E8M0 scale bytes uint8 [N, K/32]; returns bf16 [T, N].  See
    moe_linear_mxfp4 in include/moe_glue.h."""
    torch = _torch()
    _need_gpu("x", x, torch.bfloat16, 2)
    T, K = x.shape
    if K % 32 != 0:
        raise MoEGlueArgumentError(2, f"K={K} is not a multiple of the 32-column block")
    if w is None or w.dim() != 2:
        _need_gpu("w", w, None, 2)
    N = w.shape[0]
    _check_shape("w", w, torch.uint8, (N, K // 2), x.device)
    _check_shape("scales", scales, torch.uint8, (N, K // 32), x.device)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
    else:
        _check_shape("out", out, torch.bfloat16, (T, N), x.device)
    _enqueue("moe_linear_mxfp4", x.device, x.data_ptr(), T, K, w.data_ptr(), scales.data_ptr(), N, out.data_ptr())
    return out


def copy_probe(src, dst) -> None:
    """Plain 16-byte-per-lane copy of src's bytes into dst (bandwidth measuring stick)."""
    _need_gpu("src", src)
    _need_gpu("dst", dst)
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise MoEGlueArgumentError(2, "dst is smaller than src")
    check(load().moe_copy_probe(_ptr(src), _ptr(dst), nbytes, _stream(src.device)), "moe_copy_probe")


def mix_probe(src, dst, cycles: int, reads: int, writes: int, vectors_per_lane: int = 1, threads: int = 256) -> None:
    """Streaming probe: `cycles` cycles of `reads` reading and `writes`
    writing waves, vectors_per_lane KiB each (the bandwidth of that
    read:write mix)."""
    kib = 1024 * vectors_per_lane
    if reads > 0:
        _need_gpu("src", src)
        if src.numel() * src.element_size() < cycles * reads * kib:
            raise MoEGlueArgumentError(1, "src is smaller than cycles * reads * vectors_per_lane KiB")
    _need_gpu("dst", dst)
    if dst.numel() * dst.element_size() < max(cycles * writes * kib, 1024):
        raise MoEGlueArgumentError(2, "dst is smaller than cycles * writes * vectors_per_lane KiB (1 KiB at least)")
    check(load().moe_mix_probe(_ptr(src) if reads > 0 else None, _ptr(dst), cycles, reads, writes, vectors_per_lane,
                               threads, _stream(dst.device)), "moe_mix_probe")
