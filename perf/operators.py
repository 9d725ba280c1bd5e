"""Measured cases of the operators around a linear-attention layer.

  lin_fwd   chunked linear attention with one decay per head (prompts, training forward)
  lin_bwd   its gradients
  lin_step  its recurrent form for one token per sequence
  norm      RMS norm with the residual's addition; output in the input's type or in 8 bits with a scale per row
  norm_bwd  its gradients
  w4        product of a few rows with 4-bit weights and group scales

With `own` false run() computes them from elementary torch operations in 32 bits; with
`own` true it calls the package's entry points.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPE = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
_DIMS = (32, 64, 128)


def listed():
    return [
        # the training sequence of the benchmark: one sequence of 32768 tokens, 16 heads of 128
        dict(name="lin_fwd_32k", op="lin_fwd", B=1, T=32768, H=16, dk=128, dv=128, dtype="bf16", ragged=0.0, state=False),
        # a padded batch of eight prompts of odd lengths, each continued from a state
        dict(name="lin_fwd_ragged", op="lin_fwd", B=8, T=1021, H=16, dk=64, dv=128, dtype="bf16", ragged=0.8, state=True),
        # the backward pass of the training sequence
        dict(name="lin_bwd_32k", op="lin_bwd", B=1, T=32768, H=16, dk=128, dv=128, dtype="bf16", ragged=0.0, state=False),
        # a small fp32 training batch with an odd length, gradients of the state included
        dict(name="lin_bwd_f32", op="lin_bwd", B=2, T=777, H=4, dk=64, dv=64, dtype="f32", ragged=0.3, state=True),
        # one sequence, one layer, one token: latency
        dict(name="lin_step_1", op="lin_step", n=1, H=16, dk=128, dv=128, dtype="bf16"),
        # 64 sequences x 24 layers in one launch: the serving batch
        dict(name="lin_step_1536", op="lin_step", n=1536, H=16, dk=128, dv=128, dtype="bf16"),
        # a decode batch of eight tokens on the way into a projection with 8-bit inputs
        dict(name="norm_q8_8", op="norm", n=8, D=2048, dtype="bf16", residual=True, quant=True),
        # every token of the training sequence, d_model 2048
        dict(name="norm_32k", op="norm", n=32768, D=2048, dtype="bf16", residual=True, quant=False),
        # the backward pass over an odd number of tokens
        dict(name="norm_bwd_8191", op="norm_bwd", n=8191, D=2048, dtype="bf16", residual=True),
        # a small fp32 one
        dict(name="norm_bwd_f32", op="norm_bwd", n=515, D=1000, dtype="f32", residual=False),
        # one token through the projection to q, k and v of 16 heads of 128
        dict(name="w4_qkv_1", op="w4", n=1, K=2048, O=6144, group=128, dtype="bf16"),
        # eight tokens in 8 bits through a wide projection with an odd number of outputs
        dict(name="w4_wide_8", op="w4", n=8, K=2048, O=50257, group=64, dtype="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lin_fwd", "lin_bwd", "lin_step", "norm", "norm_bwd", "w4"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("lin_fwd", "lin_bwd"):
        T = _log(rng, 1, 20000 if dtype == "bf16" else 4000)
        B = _log(rng, 1, max(1, min(16, 20000 // T)))
        return dict(op=op, B=B, T=T, H=rng.randint(1, 16), dk=rng.choice(_DIMS), dv=rng.choice(_DIMS), dtype=dtype,
                    ragged=rng.choice((0.0, round(rng.uniform(0.1, 1.0), 3))), state=rng.random() < 0.5)
    if op == "lin_step":
        return dict(op=op, n=_log(rng, 1, 1200), H=rng.randint(1, 16), dk=rng.choice(_DIMS), dv=rng.choice(_DIMS), dtype=dtype)
    if op == "norm":
        return dict(op=op, n=_log(rng, 1, 20000), D=8 * _log(rng, 4, 512), dtype=dtype, residual=rng.random() < 0.5,
                    quant=rng.random() < 0.5)
    if op == "norm_bwd":
        return dict(op=op, n=_log(rng, 1, 12000), D=8 * _log(rng, 4, 512), dtype=dtype, residual=rng.random() < 0.5)
    return dict(op=op, n=_log(rng, 1, 40), K=128 * _log(rng, 1, 64), O=_log(rng, 16, 20000), group=rng.choice((32, 64, 128)),
                dtype=rng.choice(("bf16", "f32", "e4m3")))


def _lengths(case):
    """Valid tokens of each sequence: from T down by the ragged share, the last one shortest."""
    B, T = case["B"], case["T"]
    return [T - int(T * case["ragged"] * b / max(1, B - 1)) if B > 1 else T - int(T * case["ragged"] * 0.5) for b in range(B)]


def work(case):
    op, s = case["op"], {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    if op in ("lin_fwd", "lin_bwd"):
        H, dk, dv, tok, rows = case["H"], case["dk"], case["dv"], sum(_lengths(case)), case["B"] * case["T"]
        states = case["B"] * H * dk * dv * 4
        if op == "lin_fwd":
            return {"bytes": H * s * (tok * (2 * dk + dv) + rows * dv) + states * (2 if case["state"] else 1),
                    "flops": 4 * dk * dv * H * tok}
        return {"bytes": H * s * (tok * (2 * dk + 2 * dv) + rows * (2 * dk + dv)) + states * (3 if case["state"] else 1),
                "flops": 10 * dk * dv * H * tok}
    if op == "lin_step":
        r = case["n"] * case["H"]
        return {"bytes": r * (2 * case["dk"] * case["dv"] * 4 + s * 2 * (case["dk"] + case["dv"])),
                "flops": r * 5 * case["dk"] * case["dv"]}
    if op == "norm":
        n, D = case["n"], case["D"]
        out = 1 if case["quant"] else s
        return {"bytes": n * D * (s + out + (2 * s if case["residual"] else 0)) + 4 * D + 4 * n * (2 if case["quant"] else 1),
                "flops": n * D * 5}
    if op == "norm_bwd":
        n, D = case["n"], case["D"]
        return {"bytes": n * D * s * (4 if case["residual"] else 3) + 4 * n + 8 * D, "flops": n * D * 9}
    n, K, O = case["n"], case["K"], case["O"]
    return {"bytes": O * K // 2 + 2 * O * K // case["group"] + n * K * s + n * O * (4 if case["dtype"] == "f32" else 2),
            "flops": 2 * n * K * O}


# ---- inputs -------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _unit(g, *shape):
    x = torch.nn.functional.silu(_normal(g, *shape))
    return x / x.square().sum(-1, keepdim=True).sqrt()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"op": op}
    dt = _TYPE[case["dtype"]]
    if op in ("lin_fwd", "lin_bwd", "lin_step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        lead = (case["n"],) if op == "lin_step" else (case["B"], case["T"])
        st["q"], st["k"] = _unit(g, *lead, H, dk).to(dt), _unit(g, *lead, H, dk).to(dt)
        st["v"] = _normal(g, *lead, H, dv).to(dt)
        # one decay rate per head, log-uniform in [1e-4, 0.7]
        u = torch.rand(H, generator=g, device="cuda")
        st["log_decay"] = -(1e-4 * (0.7 / 1e-4) ** u)
        st["scale"] = 1.0 / math.sqrt(dk)
        if op == "lin_step":
            st["S"] = _normal(g, *lead, H, dk, dv)
            return st
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        st["S0"] = _normal(g, lead[0], H, dk, dv) if case["state"] else None
        if op == "lin_bwd":
            st["dy"] = _normal(g, *lead, H, dv).to(dt)
            st["dS_T"] = _normal(g, lead[0], H, dk, dv) if case["state"] else None
        return st
    if op in ("norm", "norm_bwd"):
        n, D = case["n"], case["D"]
        st["x"] = _normal(g, n, D).to(dt)
        st["residual"] = (4.0 * _normal(g, n, D)).to(dt) if case["residual"] else None
        st["weight"] = 1.0 + 0.1 * _normal(g, D)
        st["eps"] = 1e-6
        if op == "norm":
            st["quant"] = case["quant"]
            return st
        # the backward pass has the residual stream and the norm's rstd in hand from the forward pass
        st["h"] = st.pop("x") if st["residual"] is None else (st.pop("x").float() + st["residual"].float()).to(dt)
        st.pop("residual")
        st["rstd"] = torch.rsqrt(st["h"].double().square().mean(-1) + st["eps"]).float()
        st["dy"] = _normal(g, n, D).to(dt)
        st["dh"] = _normal(g, n, D).to(dt) if case["residual"] else None
        return st
    n, K, O, G = case["n"], case["K"], case["O"], case["group"]
    codes = torch.randint(0, 16, (O, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(O, K // G, generator=g, device="cuda")) / (4.0 * math.sqrt(K))).to(BF16)
    st["wq"], st["ws"] = _w4_layout(codes, scales)
    st["O"] = O
    x = _normal(g, n, K)
    st["x_scale"] = None
    if dt == E4M3:
        st["x_scale"] = x.abs().amax(-1) / 448.0
        x = x / st["x_scale"][:, None]
    st["x"] = x.to(dt)
    return st


# The 4-bit weight layout: tiles of 16 outputs x 128 inputs, 1024 bytes each. Lane (g, t),
# g = 0..7, t = 0..3, has 32 bytes: for the outputs g and g + 8, four 4-byte words
# j = 0..3, word j holding the inputs 32 j + 8 t .. + 7, lowest nibble first. Scales:
# bf16, for each tile and each group of its inputs the 16 outputs' scales.
def _w4_layout(codes, scales):
    O, K = codes.shape
    pad = -O % 16
    c = torch.nn.functional.pad(codes, (0, 0, 0, pad), value=8).view(-1, 2, 8, K // 128, 4, 4, 4, 2)
    # tile, half, g, block, j, t, byte, nibble -> tile, block, g, t, half, j, byte, nibble
    c = c.permute(0, 3, 2, 5, 1, 4, 6, 7)
    wq = (c[..., 0] | (c[..., 1] << 4)).reshape(-1, K // 128, 1024).contiguous()
    gpb = scales.shape[1] * 128 // K
    s = torch.nn.functional.pad(scales, (0, 0, 0, pad)).view(-1, 16, K // 128, gpb)
    return wq, s.permute(0, 2, 3, 1).contiguous()


def _w4_values(wq, ws, O, dtype):
    tiles, blocks = wq.shape[:2]
    c = torch.stack((wq & 15, wq >> 4), -1).view(tiles, blocks, 8, 4, 2, 4, 4, 2)
    c = c.permute(0, 4, 2, 1, 5, 3, 6, 7).reshape(tiles * 16, blocks * 128)[:O]
    s = ws.permute(0, 3, 1, 2).reshape(tiles * 16, -1)[:O]
    return (c.to(dtype) - 8.0) * s.to(dtype).repeat_interleave(c.shape[1] // s.shape[1], 1)


# ---- plain forms ----------------------------------------------------------------


def _chunks(x, keep, n, C):
    """[B,T,H,d] -> [B,H,n,C,d] in 32 bits, zeros at padded tokens."""
    x = torch.where(keep[:, :, None, None], x.float(), 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - x.shape[1]))
    return x.view(x.shape[0], n, C, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4)


def _tokens(x, T, keep, dtype):
    """[B,H,n,C,d] -> [B,T,H,d], zeros at padded tokens."""
    B, H, n, C, d = x.shape
    x = x.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, d)[:, :T]
    return torch.where(keep[:, :, None, None], x, 0.0).to(dtype)


def _power(ld, e, ok=None):
    """decay^e in 32 bits from 64, zero where not ok; ld broadcasts against e."""
    p = torch.exp(ld.double() * e.double())
    return (p if ok is None else torch.where(ok, p, 0.0)).float()


def _lin_setup(st):
    B, T = st["q"].shape[:2]
    dev, C = st["q"].device, 128
    n = max(1, -(-T // C))
    lens = torch.full((B,), T, device=dev) if st["lengths"] is None else st["lengths"].long()
    keep = torch.arange(T, device=dev)[None] < lens[:, None]
    ld, i, c = st["log_decay"], torch.arange(C, device=dev), torch.arange(n, device=dev)
    D = _power(ld[:, None, None], (i[:, None] - i[None]).clamp(min=0), i[:, None] >= i[None])  # [H,C,C]
    before = c[:, None] > c[None]
    W = _power(ld[:, None, None], ((c[:, None] - c[None] - 1) * C).clamp(min=0), before)  # [H,n,n]
    up = _power(ld[:, None], i + 1)[None, :, None, :, None]
    down = _power(ld[:, None], C - 1 - i)[None, :, None, :, None]
    t = torch.arange(n * C, device=dev)
    left = lens[:, None] - 1 - t[None]  # tokens after this one
    end = _power(ld[None, :, None], left[:, None].clamp(min=0), (left >= 0)[:, None]).view(B, -1, n, C, 1)
    whole = _power(ld[None], lens[:, None])[:, :, None, None]
    into = _power(ld[:, None], c * C)[None, :, :, None, None]
    return n, C, keep, D, W, up, down, end, whole, into


def _lin_states(W, U, S0, into):
    """States entering each chunk from the chunks' contributions U [B,H,n,dk,dv]."""
    S = (W @ U.flatten(3)).view_as(U)
    return S if S0 is None else S + into * S0[:, :, None]


def _lin_fwd_plain(st):
    n, C, keep, D, W, up, down, end, whole, into = _lin_setup(st)
    q, k, v = (_chunks(st[x], keep, n, C) for x in "qkv")
    S0 = st["S0"]
    S = _lin_states(W, (k * down).mT @ v, S0, into)
    y = ((q @ k.mT) * D[None, :, None]) @ v + (q * up) @ S
    S_T = (k * end).flatten(2, 3).mT @ v.flatten(2, 3)
    if S0 is not None:
        S_T = S_T + whole * S0
    return {"y": _tokens(st["scale"] * y, st["q"].shape[1], keep, st["v"].dtype), "S_T": S_T}


def _lin_bwd_plain(st):
    n, C, keep, D, W, up, down, end, whole, into = _lin_setup(st)
    q, k, v, dy = (_chunks(st[x], keep, n, C) for x in ("q", "k", "v", "dy"))
    dy = dy * st["scale"]
    T, S0, dS_T = st["q"].shape[1], st["S0"], st["dS_T"]
    S = _lin_states(W, (k * down).mT @ v, S0, into)
    G = (q * up).mT @ dy  # cotangent of the state entering each chunk, from that chunk
    R = (W.mT @ G.flatten(3)).view_as(G)  # and of the state leaving it, from later chunks
    P, dP = (q @ k.mT) * D[None, :, None], (dy @ v.mT) * D[None, :, None]
    dq = dP @ k + up * (dy @ S.mT)
    dk = dP.mT @ q + down * (v @ R.mT)
    dv = P.mT @ dy + down * (k @ R)
    dS0 = G[:, :, 0] + _power(st["log_decay"], torch.tensor(C, device=q.device))[None, :, None, None] * R[:, :, 0]
    if dS_T is not None:
        dk = dk + end * (v @ dS_T[:, :, None].mT)
        dv = dv + end * (k @ dS_T[:, :, None])
        dS0 = dS0 + whole * dS_T
    out = {m: _tokens(x, T, keep, st["q"].dtype) for m, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    return {**out, "dS0": dS0}


def _lin_step_plain(st):
    S, q, k, v = st["S"], st["q"].float(), st["k"].float(), st["v"].float()
    S.mul_(torch.exp(st["log_decay"].double()).float()[None, :, None, None]).add_(k[..., None] * v[..., None, :])  # in place
    return {"y": (st["scale"] * (q[..., None] * S).sum(-2)).to(st["v"].dtype), "S": S}


def _norm_plain(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    rstd = torch.rsqrt(h.square().mean(-1) + st["eps"])
    y = h * rstd[:, None] * st["weight"]
    out = {"rstd": rstd} if st["residual"] is None else {"rstd": rstd, "h": h.to(st["x"].dtype)}
    if not st["quant"]:
        return {**out, "y": y.to(st["x"].dtype)}
    top = y.abs().amax(-1)
    q = y * torch.where(top > 0, 448.0 / top, 0.0)[:, None]
    return {**out, "q": q.clamp(-448.0, 448.0).to(E4M3), "scale": top / 448.0}


def _norm_bwd_plain(st):
    xh = st["h"].float() * st["rstd"][:, None]
    dy = st["dy"].float()
    g = dy * st["weight"]
    dx = st["rstd"][:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(st["h"].dtype), "dweight": (dy * xh).sum(0)}


def _w4_plain(st):
    x = st["x"].float()
    if st["x_scale"] is not None:
        x = x * st["x_scale"][:, None]
    return {"y": (x @ _w4_values(st["wq"], st["ws"], st["O"], F32).mT).to(F32 if st["x"].dtype == F32 else BF16)}


_PLAIN = {"lin_fwd": _lin_fwd_plain, "lin_bwd": _lin_bwd_plain, "lin_step": _lin_step_plain, "norm": _norm_plain,
          "norm_bwd": _norm_bwd_plain, "w4": _w4_plain}


# ---- the framework's calls --------------------------------------------------------


def _own(st):
    import gated_delta_rule_muir_b200 as muir
    op = st["op"]
    if op == "lin_fwd":
        y, S_T = muir.lin_attn_fwd(st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"], lengths=st["lengths"],
                                   S0=st["S0"])
        return {"y": y, "S_T": S_T}
    if op == "lin_bwd":
        g = muir.lin_attn_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["dy"], scale=st["scale"], lengths=st["lengths"],
                              S0=st["S0"], dS_T=st["dS_T"])
        return {m: g[m] for m in ("dq", "dk", "dv", "dS0")}
    if op == "lin_step":
        y = muir.lin_attn_step(st["S"], st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"])  # S in place
        return {"y": y, "S": st["S"]}
    if op == "norm":
        f = muir.rms_norm_quant if st["quant"] else muir.rms_norm
        return f(st["x"], st["weight"], residual=st["residual"], eps=st["eps"])
    if op == "norm_bwd":
        dx, dw = muir.rms_norm_bwd(st["dy"], st["h"], st["weight"], st["rstd"], dh=st["dh"])
        return {"dx": dx, "dweight": dw}
    return {"y": muir.w4_matvec(st["x"], st["wq"], st["ws"], st["O"], x_scale=st["x_scale"])}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---- 64-bit values ------------------------------------------------------------------


def _lin_exact(st, backward):
    """By the quadratic sums over all earlier tokens, a block of rows at a time."""
    q, k, v = (st[x].double().permute(0, 2, 1, 3) for x in "qkv")
    B, H, T, _ = q.shape
    dev = q.device
    lens = torch.full((B,), T, device=dev) if st["lengths"] is None else st["lengths"].long()
    pos = torch.arange(T, device=dev)
    live = (pos[None] < lens[:, None])[:, None, :, None]
    q, k, v = (x * live for x in (q, k, v))
    ld = st["log_decay"].double().view(1, H, 1, 1)
    tail = torch.exp(ld * (lens.view(B, 1, 1, 1) - 1 - pos.view(1, 1, T, 1)).clamp(min=0)) * live
    whole = torch.exp(ld * lens.view(B, 1, 1, 1))
    head = torch.exp(ld * (pos.view(1, 1, T, 1) + 1))
    S0 = None if st["S0"] is None else st["S0"].double()
    if backward:
        dy = st["dy"].double().permute(0, 2, 1, 3) * live * st["scale"]
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    else:
        y = torch.zeros_like(v)
    rows = max(1, min(T, (1 << 29) // max(1, B * H * T)))
    for a in range(0, T, rows):
        e = min(T, a + rows)
        gap = pos[a:e, None] - pos[None, :e]
        D = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), 0.0)
        P = (q[:, :, a:e] @ k[:, :, :e].mT) * D
        if not backward:
            y[:, :, a:e] = P @ v[:, :, :e]
            continue
        dv[:, :, :e] += P.mT @ dy[:, :, a:e]
        del P
        dP = (dy[:, :, a:e] @ v[:, :, :e].mT) * D
        dq[:, :, a:e] = dP @ k[:, :, :e]
        dk[:, :, :e] += dP.mT @ q[:, :, a:e]
    if not backward:
        S_T = (k * tail).mT @ v
        if S0 is not None:
            y, S_T = y + head * (q @ S0), S_T + whole * S0
        return {"y": (st["scale"] * y).permute(0, 2, 1, 3), "S_T": S_T}
    dS0 = (q * head).mT @ dy
    if S0 is not None:
        dq += head * (dy @ S0.mT)
    if st["dS_T"] is not None:
        dS_T = st["dS_T"].double()
        dk += tail * (v @ dS_T.mT)
        dv += tail * (k @ dS_T)
        dS0 = dS0 + whole * dS_T
    return {**{m: x.permute(0, 2, 1, 3) for m, x in (("dq", dq), ("dk", dk), ("dv", dv))}, "dS0": dS0}


def _e4m3_value(x):
    """The nearest e4m3 number, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op in ("lin_fwd", "lin_bwd"):
        return _lin_exact(st, op == "lin_bwd")
    if op == "lin_step":
        S = torch.exp(st["log_decay"].double())[:, None, None] * st["S"].double()
        S = S + torch.einsum("nhi,nhj->nhij", st["k"].double(), st["v"].double())
        return {"y": st["scale"] * torch.einsum("nhi,nhij->nhj", st["q"].double(), S), "S": S}
    if op == "norm":
        h = st["x"].double() + (0.0 if st["residual"] is None else st["residual"].double())
        rstd = 1.0 / torch.sqrt((h * h).sum(-1) / h.shape[-1] + st["eps"])
        y = h * rstd[:, None] * st["weight"].double()
        out = {"rstd": rstd} if st["residual"] is None else {"rstd": rstd, "h": h}
        if not st["quant"]:
            return {**out, "y": y}
        scale = y.abs().max(-1).values / 448.0
        return {**out, "q": _e4m3_value(torch.where(scale[:, None] > 0, y / scale[:, None], 0.0)), "scale": scale}
    if op == "norm_bwd":
        h, dy, r, w = st["h"].double(), st["dy"].double(), st["rstd"].double()[:, None], st["weight"].double()
        mean = torch.einsum("nd,nd,d->n", dy, h, w)[:, None] / h.shape[1]
        dx = r * dy * w - r ** 3 * mean * h
        return {"dx": dx if st["dh"] is None else dx + st["dh"].double(), "dweight": torch.einsum("nd,nd->d", dy, h * r)}
    x = st["x"].double() * (1.0 if st["x_scale"] is None else st["x_scale"].double()[:, None])
    w = _w4_values(st["wq"], st["ws"], st["O"], torch.float64)
    return {"y": torch.einsum("nk,ok->no", x, w)}
