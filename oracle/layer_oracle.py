"""fp64 CPU oracle of the operators around the state update (test infrastructure):
linear attention with one decay per head, RMS norm, 4-bit products. Written from the
definitions, token by token; no code is shared with the CUDA path. The `_abs`
results are the same sums over absolute values, the scale of their rounding errors."""
import numpy as np


def lin_forward(q, k, v, log_decay, scale=1.0, lengths=None, S0=None):
    """q, k [B,T,H,dk], v [B,T,H,dv], log_decay [H] -> y [B,T,H,dv], S_T [B,H,dk,dv]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    lam = np.exp(log_decay)[:, None, None]
    y = np.zeros((B, T, H, dv))
    S_T = np.zeros((B, H, dk, dv))
    for b in range(B):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        for t in range(T if lengths is None else min(T, max(0, int(lengths[b])))):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            y[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], S)
        S_T[b] = S
    return y, S_T


def lin_backward(q, k, v, log_decay, dy, scale=1.0, lengths=None, S0=None, dS_T=None):
    """Gradients by the reverse recurrence: dS_t = scale q_t dy_t^T + lambda dS_{t+1}."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    lam = np.exp(log_decay)[:, None, None]
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dS0": np.zeros((B, H, dk, dv))}
    for b in range(B):
        n = T if lengths is None else min(T, max(0, int(lengths[b])))
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        for t in range(n):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            g["dq"][b, t] = scale * np.einsum("hij,hj->hi", S, dy[b, t])
        dS = np.zeros((H, dk, dv)) if dS_T is None else dS_T[b].copy()
        for t in range(n - 1, -1, -1):
            dS = dS + scale * q[b, t][:, :, None] * dy[b, t][:, None, :]
            g["dk"][b, t] = np.einsum("hij,hj->hi", dS, v[b, t])
            g["dv"][b, t] = np.einsum("hij,hi->hj", dS, k[b, t])
            dS = lam * dS
        g["dS0"][b] = dS
    return g


def lin_forward_abs(q, k, v, log_decay, scale=1.0, lengths=None, S0=None):
    return lin_forward(abs(q), abs(k), abs(v), log_decay, abs(scale), lengths, None if S0 is None else abs(S0))


def lin_backward_abs(q, k, v, log_decay, dy, scale=1.0, lengths=None, S0=None, dS_T=None):
    return lin_backward(abs(q), abs(k), abs(v), log_decay, abs(dy), abs(scale), lengths, None if S0 is None else abs(S0),
                        None if dS_T is None else abs(dS_T))


def rms_norm(x, weight, residual=None, eps=1e-6):
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1) + eps)
    return h * rstd[:, None] * weight, h, rstd


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    xh, g = h * rstd[:, None], dy * weight
    dx = rstd[:, None] * (g - xh * np.mean(g * xh, axis=-1, keepdims=True))
    return (dx if dh is None else dx + dh), np.sum(dy * xh, axis=0)


def e4m3(x):
    """The nearest e4m3 number (largest 448), ties to the even one."""
    a = np.maximum(np.abs(x), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(a)) - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0)


def w4_dequantize(codes, scales):
    """codes [O,K] 0..15, scales [O,K/group] -> weights [O,K]."""
    group = codes.shape[1] // scales.shape[1]
    return (codes.astype(np.float64) - 8.0) * np.repeat(scales, group, axis=1)


def w4_layout(codes, scales):
    """The packed layout, byte by byte from its description."""
    O, K = codes.shape
    tiles, blocks, gpb = (O + 15) // 16, K // 128, scales.shape[1] * 128 // K
    wq = np.zeros((tiles, blocks, 1024), np.uint8)
    ws = np.zeros((tiles, blocks, gpb, 16))
    for tile in range(tiles):
        for kb in range(blocks):
            for byte in range(1024):
                lane, rest = divmod(byte, 32)
                half, rest = divmod(rest, 16)
                j, pair = divmod(rest, 4)
                g, t = divmod(lane, 4)
                o, k = tile * 16 + half * 8 + g, kb * 128 + 32 * j + 8 * t + 2 * pair
                lo, hi = (codes[o, k], codes[o, k + 1]) if o < O else (8, 8)
                wq[tile, kb, byte] = (lo & 15) | ((hi & 15) << 4)
            for gr in range(gpb):
                for o16 in range(16):
                    o = tile * 16 + o16
                    ws[tile, kb, gr, o16] = scales[o, kb * gpb + gr] if o < O else 0.0
    return wq, ws
