"""The operators around the state update: linear attention with one decay per head,
RMS norm with the residual's addition, products with 4-bit weights.

As in the rest of the binding, each function only checks shapes, dtypes and
devices, allocates outputs and workspace with torch, and calls the C ABI
(include/muir.h). Work goes to `stream` (default: the current stream of the
operands' device); what a call allocates is allocated for that stream.
"""
from __future__ import annotations

import ctypes as C
import functools
import inspect

import torch

from . import _native as N

_E4M3 = torch.float8_e4m3fn
# handle of a device's current stream (a tenth of a microsecond; building a Stream object takes three)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, shape, dtype, device):
    if type(t) is not torch.Tensor and not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: must be a contiguous CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other operands on {device}")


def _dims(t, name, n):
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _int32(name, size):
    """Sizes that the C ABI holds in 32 bits: a larger one would reach it cut to its low bits."""
    if size > 0x7fffffff:
        raise ValueError(f"{name} must be below 2^31, got {size}")


def _io_code(t, name):
    code = {torch.float32: N.MUIR_F32, torch.bfloat16: N.MUIR_BF16}.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return code


def _placed(fn):
    """Runs fn with `stream` (default: the current stream of the first operand's device) as a raw
    handle, that device and stream being current for its allocations and launches. The common
    call, the current device and its current stream, switches nothing."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        t = args[0] if args else kw.get(first)
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{first}: expected a tensor, got {type(t).__name__}")
        if not t.is_cuda:
            return fn(*args, stream=0, **kw)  # which refuses it
        index = t.get_device()
        if stream is None:
            if index == torch.cuda.current_device():
                return fn(*args, stream=_raw_stream(index), **kw)
            stream = torch.cuda.current_stream(index)
        elif stream.device_index != index:
            raise ValueError(f"stream of {stream.device}, operands on {t.device}")
        with torch.cuda.device(index), torch.cuda.stream(stream):
            return fn(*args, stream=stream.cuda_stream, **kw)
    return call


def _workspace(nbytes, device, ws):
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    if not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    return ws


def _like(t, name, x):
    """The output `name`, shaped and typed like x."""
    if t is None:
        return torch.empty_like(x)
    _need(t, name, x.shape, x.dtype, x.device)
    return t


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, shape, dtype, device)
    return t


def _lin_args(q, k, v, log_decay, scale, lengths, S0):
    B, T, H, dk = _dims(q, "q", 4)
    dv = _dims(v, "v", 4)[3]
    _int32("a number of heads or channels", max(H, dk, dv))
    dev = q.device
    code = _io_code(q, "q")
    _need(q, "q", (B, T, H, dk), q.dtype, dev)
    _need(k, "k", (B, T, H, dk), q.dtype, dev)
    _need(v, "v", (B, T, H, dv), q.dtype, dev)
    _need(log_decay, "log_decay", (H,), torch.float32, dev)
    if lengths is not None:
        _need(lengths, "lengths", (B,), torch.int32, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    a = N.LinArgs(B, T, H, dk, dv, code, 0, float(scale), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                  _ptr(lengths), _ptr(S0))
    return a, (B, T, H, dk, dv, q.dtype, dev)


def lin_attn_workspace_bytes(q, k, v, log_decay, *, backward=False) -> int:
    """Bytes of workspace that lin_attn_fwd (or lin_attn_bwd) needs for operands of these sizes."""
    a, _ = _lin_args(q, k, v, log_decay, 1.0, None, None)
    lib = N.load()
    return int((lib.muir_lin_bwd_workspace if backward else lib.muir_lin_fwd_workspace)(C.byref(a)))


@_placed
def lin_attn_fwd(q, k, v, log_decay, *, scale=1.0, lengths=None, S0=None, want_state=True, y=None, S_T=None,
                 workspace=None, stream=None):
    """Linear attention with one decay per head, S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,
    y_t = scale S_t^T q_t, over whole sequences: q, k [B,T,H,dk], v [B,T,H,dv] (fp32 or bf16),
    log_decay [H] fp32 (<= 0), lengths [B] int32 (valid tokens of a padded batch), S0
    [B,H,dk,dv] fp32. Returns (y [B,T,H,dv], S_T [B,H,dk,dv] fp32 or None); y is zero at padded
    tokens and S_T is the state after the last valid one. The decays are constants: they get
    no gradient. bf16 operands are multiplied on the tensor cores, with one bf16 rounding of
    the token-token weights and of the state that y reads; fp32 operands at fp32 accuracy."""
    a, (B, T, H, dk, dv, dt, dev) = _lin_args(q, k, v, log_decay, scale, lengths, S0)
    lib = N.load()
    y = _like(y, "y", v)
    S_T = _out(S_T, "S_T", (B, H, dk, dv), torch.float32, dev) if want_state else None
    nbytes = int(lib.muir_lin_fwd_workspace(C.byref(a)))
    ws = _workspace(nbytes, dev, workspace)
    N.check(lib.muir_lin_fwd(C.byref(a), _ptr(y), _ptr(S_T), _ptr(ws), nbytes, stream), "muir_lin_fwd")
    return y, S_T


@_placed
def lin_attn_bwd(q, k, v, log_decay, dy, *, scale=1.0, lengths=None, S0=None, dS_T=None, want_dS0=True, outputs=None,
                 workspace=None, stream=None):
    """Gradients of lin_attn_fwd: a dict of dq, dk, dv (shaped and typed like q, k, v) and dS0
    [B,H,dk,dv] fp32 (None if not wanted). `outputs` (a dict from an earlier call) is reused."""
    a, (B, T, H, dk, dv, dt, dev) = _lin_args(q, k, v, log_decay, scale, lengths, S0)
    _need(dy, "dy", (B, T, H, dv), dt, dev)
    if dS_T is not None:
        _need(dS_T, "dS_T", (B, H, dk, dv), torch.float32, dev)
    lib = N.load()
    o = outputs or {}
    out = {"dq": _like(o.get("dq"), "dq", q), "dk": _like(o.get("dk"), "dk", k),
           "dv": _like(o.get("dv"), "dv", v),
           "dS0": _out(o.get("dS0"), "dS0", (B, H, dk, dv), torch.float32, dev) if want_dS0 else None}
    g = N.LinGrads(dy.data_ptr(), _ptr(dS_T), *(_ptr(out[n]) for n in ("dq", "dk", "dv", "dS0")))
    nbytes = int(lib.muir_lin_bwd_workspace(C.byref(a)))
    ws = _workspace(nbytes, dev, workspace)
    N.check(lib.muir_lin_bwd(C.byref(a), C.byref(g), _ptr(ws), nbytes, stream), "muir_lin_bwd")
    return out


@_placed
def lin_attn_step(S, q, k, v, log_decay, *, scale=1.0, y=None, stream=None):
    """One token of lin_attn_fwd for n sequences: S [n,H,dk,dv] fp32 updated in place, q, k
    [n,H,dk], v [n,H,dv]. Returns y [n,H,dv]."""
    n, H, dk, dv = _dims(S, "S", 4)
    _int32("a number of heads or channels", max(H, dk, dv))
    dev = S.device
    code = _io_code(q, "q")
    _need(S, "S", (n, H, dk, dv), torch.float32, dev)
    for name, t, d in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        _need(t, name, (n, H, d), q.dtype, dev)
    _need(log_decay, "log_decay", (H,), torch.float32, dev)
    lib = N.load()
    y = _like(y, "y", v)
    a = N.LinStepArgs(n, H, dk, dv, code, float(scale), S.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                      log_decay.data_ptr(), y.data_ptr())
    N.check(lib.muir_lin_step(C.byref(a), stream), "muir_lin_step")
    return y


def _norm_operands(x, weight, residual):
    n, d = _dims(x, "x", 2)
    _int32("d", d)
    dev = x.device
    code = _io_code(x, "x")
    _need(x, "x", (n, d), x.dtype, dev)
    _need(weight, "weight", (d,), torch.float32, dev)
    if residual is not None:
        _need(residual, "residual", (n, d), x.dtype, dev)
    return n, d, dev, code


@_placed
def rms_norm(x, weight, *, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """RMS norm of rows x [n,d] (fp32 or bf16), weight [d] fp32, with the residual's addition:
    h = x + residual, y = h (mean h^2 + eps)^(-1/2) weight. Returns a dict of y, rstd [n] fp32
    and, with a residual, h (the new residual stream; may be the residual's own buffer)."""
    n, d, dev, code = _norm_operands(x, weight, residual)
    lib = N.load()
    out = {"y": _like(y, "y", x), "rstd": _out(rstd, "rstd", (n,), torch.float32, dev)}
    if residual is not None:
        out["h"] = _like(h, "h", x)
    N.check(lib.muir_rms_norm(_ptr(x), _ptr(residual), _ptr(weight), _ptr(out["y"]), _ptr(out.get("h")), _ptr(out["rstd"]),
                              n, d, float(eps), code, stream), "muir_rms_norm")
    return out


@_placed
def rms_norm_quant(x, weight, *, residual=None, eps=1e-6, q=None, scale=None, h=None, rstd=None, stream=None):
    """rms_norm with its output in 8 bits: q [n,d] float8_e4m3fn and scale [n] fp32, q scale ~ y,
    scale = max |y| / 448 of the row. Returns a dict of q, scale, rstd and, with a residual, h."""
    n, d, dev, code = _norm_operands(x, weight, residual)
    lib = N.load()
    out = {"q": _out(q, "q", (n, d), _E4M3, dev), "scale": _out(scale, "scale", (n,), torch.float32, dev),
           "rstd": _out(rstd, "rstd", (n,), torch.float32, dev)}
    if residual is not None:
        out["h"] = _like(h, "h", x)
    N.check(lib.muir_rms_norm_quant(_ptr(x), _ptr(residual), _ptr(weight), _ptr(out["q"]), _ptr(out["scale"]),
                                    _ptr(out.get("h")), _ptr(out["rstd"]), n, d, float(eps), code, stream),
            "muir_rms_norm_quant")
    return out


@_placed
def rms_norm_bwd(dy, h, weight, rstd, *, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of rms_norm from its h (its x, without a residual) and rstd: (dx [n,d], dweight
    [d] fp32). dx is the gradient of x and of the residual alike; dh is the cotangent of h."""
    n, d = _dims(h, "h", 2)
    _int32("d", d)
    dev = h.device
    code = _io_code(h, "h")
    _need(h, "h", (n, d), h.dtype, dev)
    _need(dy, "dy", (n, d), h.dtype, dev)
    _need(weight, "weight", (d,), torch.float32, dev)
    _need(rstd, "rstd", (n,), torch.float32, dev)
    if dh is not None:
        _need(dh, "dh", (n, d), h.dtype, dev)
    lib = N.load()
    dx = _like(dx, "dx", h)
    dweight = _out(dweight, "dweight", (d,), torch.float32, dev)
    nbytes = int(lib.muir_rms_norm_bwd_workspace(n, d))
    ws = _workspace(nbytes, dev, workspace)
    N.check(lib.muir_rms_norm_bwd(_ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd), _ptr(dh), _ptr(dx), _ptr(dweight), n, d,
                                  code, _ptr(ws), nbytes, stream), "muir_rms_norm_bwd")
    return dx, dweight


@_placed
def w4_quantize(w, *, group=128, stream=None):
    """Weights [O,K] (fp32 or bf16) to 4 bits: (codes [O,K] uint8 in 0..15, scales [O,K/group]
    bf16), w ~ scale (code - 8), scale = max |w| / 7 of each group."""
    O, K = _dims(w, "w", 2)
    _int32("O and K", max(O, K))
    dev = w.device
    code = _io_code(w, "w")
    _need(w, "w", (O, K), w.dtype, dev)
    if group not in (32, 64, 128) or K % 128:
        raise ValueError(f"group must be 32, 64 or 128 and K a multiple of 128 (got {group}, {K})")
    lib = N.load()
    codes = torch.empty(O, K, dtype=torch.uint8, device=dev)
    scales = torch.empty(O, K // group, dtype=torch.bfloat16, device=dev)
    N.check(lib.muir_w4_quantize(_ptr(w), _ptr(codes), _ptr(scales), K, O, group, code, stream), "muir_w4_quantize")
    return codes, scales


@_placed
def w4_pack(codes, scales, *, stream=None):
    """Codes [O,K] uint8 and scales [O,K/group] bf16 in the layout of w4_matvec: (wq uint8
    [ceil(O/16), K/128, 1024], ws bf16 [ceil(O/16), K/128, 128/group, 16]); see include/muir.h."""
    O, K = _dims(codes, "codes", 2)
    _int32("O and K", max(O, K))
    ng = _dims(scales, "scales", 2)[1]
    dev = codes.device
    if K % 128 or ng == 0 or K % ng or K // ng not in (32, 64, 128):
        raise ValueError(f"K must be a multiple of 128 in groups of 32, 64 or 128 (got K={K}, {ng} groups)")
    group = K // ng
    _need(codes, "codes", (O, K), torch.uint8, dev)
    _need(scales, "scales", (O, ng), torch.bfloat16, dev)
    lib = N.load()
    tiles = (O + 15) // 16
    wq = torch.empty(tiles, K // 128, 1024, dtype=torch.uint8, device=dev)
    ws = torch.empty(tiles, K // 128, 128 // group, 16, dtype=torch.bfloat16, device=dev)
    N.check(lib.muir_w4_pack(_ptr(codes), _ptr(scales), _ptr(wq), _ptr(ws), K, O, group, stream), "muir_w4_pack")
    return wq, ws


@_placed
def w4_matvec(x, wq, ws, O, *, x_scale=None, out_dtype=None, y=None, stream=None):
    """y [n,O] = x [n,K] times the transposed 4-bit weights (wq, ws of w4_pack, O outputs). x:
    fp32 or bf16 (y of the same type), or float8_e4m3fn with x_scale [n] fp32, as rms_norm_quant
    gives them (y bf16, or fp32 by out_dtype). Meant for few rows: weights are read once per 32."""
    n, K = _dims(x, "x", 2)
    _int32("O and K", max(O, K))
    dev = x.device
    tiles, blocks, _ = _dims(wq, "wq", 3)
    gpb = _dims(ws, "ws", 4)[2]
    if gpb not in (1, 2, 4):
        raise ValueError(f"ws: expected 1, 2 or 4 groups per block of 128 inputs, got {gpb}")
    if K != blocks * 128 or not 0 < O <= tiles * 16 or O <= (tiles - 1) * 16:
        raise ValueError(f"wq holds {blocks * 128} inputs and {tiles} tiles of 16 outputs; got K={K}, O={O}")
    eight = x.dtype == _E4M3
    code = N.MUIR_E4M3 if eight else _io_code(x, "x")
    ydt = (out_dtype or torch.bfloat16) if eight else x.dtype
    if out_dtype not in (None, ydt) or ydt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out_dtype {out_dtype} with x of {x.dtype}")
    _need(x, "x", (n, K), x.dtype, dev)
    _need(wq, "wq", (tiles, blocks, 1024), torch.uint8, dev)
    _need(ws, "ws", (tiles, blocks, gpb, 16), torch.bfloat16, dev)
    if x_scale is not None:
        if not eight:
            raise ValueError("x_scale belongs to 8-bit rows")
        _need(x_scale, "x_scale", (n,), torch.float32, dev)
    lib = N.load()
    y = _out(y, "y", (n, O), ydt, dev)
    N.check(lib.muir_w4_matvec(_ptr(x), _ptr(x_scale), _ptr(wq), _ptr(ws), _ptr(y), n, K, O, 128 // gpb, code,
                               N.MUIR_F32 if ydt == torch.float32 else N.MUIR_BF16, stream), "muir_w4_matvec")
    return y
