"""Gradients against differences, along directions in which a wrong gradient shows: each
test asserts that what it compares stands far above its tolerance, and that leaving out a
part of the gradient would not pass."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo
from tests.test_gpu_lin_attn import _tol

pytestmark = pytest.mark.gpu


def _np(x):
    return x.double().cpu().numpy()


def test_chain_of_norm_and_attention(cuda_ok):
    """d loss / d x through attention over the norm's output, fp32, along the gradient itself.

    The difference over 2 h = 1 differs from the derivative by the chain's truncation, which
    the oracle gives in 64 bits, and by rounding: an output of the chain errs by (192 + T)
    2^-24 of its sum of absolute terms in attention and by three times (n / 16 + 24) 2^-24
    in the norm (q, k and v are its output), the gradient by as much twice over (both operators, forward
    and backward) relative to its own parts' absolute sum."""
    r = np.random.default_rng(1)
    T, H, D = 70, 2, 32
    n = H * D
    x = torch.tensor(r.normal(size=(T, n)), dtype=torch.float32).cuda()
    w = torch.tensor(1 + 0.1 * r.normal(size=n), dtype=torch.float32).cuda()
    ld = torch.tensor([-0.02, -0.5]).cuda()
    dy = torch.tensor(r.normal(size=(1, T, H, D)), dtype=torch.float32).cuda()
    xd, wd, ldd, dyd = (_np(a) for a in (x, w, ld, dy))

    def forward(x):
        f = muir.rms_norm(x, w)
        a = f["y"].view(1, T, H, D)
        return f, a, muir.lin_attn_fwd(a, a, a, ld, scale=0.05)[0]

    def forward64(x, attend=lo.lin_forward):
        a, _, rstd = lo.rms_norm(x, wd)
        a = a.reshape(1, T, H, D)
        return a, rstd, attend(a, a, a, ldd, 0.05)[0]
    f, a, y = forward(x)
    g = muir.lin_attn_bwd(a, a, a, ld, dy, scale=0.05, want_dS0=False)
    dx = {m: muir.rms_norm_bwd(g[m].view(T, n), x, w, f["rstd"])[0].double() for m in ("dq", "dk", "dv")}
    whole = (g["dq"] + g["dk"] + g["dv"]).view(T, n)
    total = muir.rms_norm_bwd(whole, x, w, f["rstd"])[0].double()
    e = (total / total.norm()).float()
    up, down = x + 0.5 * e, x - 0.5 * e
    real = up.double() - down.double()
    loss = lambda x: (forward(x)[2].double() * dy.double()).sum().item()
    loss64 = lambda x: (forward64(x)[2] * dyd).sum()
    diff, want = loss(up) - loss(down), (total * real).sum().item()
    a64, rstd64, _ = forward64(xd)
    g64 = lo.lin_backward(a64, a64, a64, ldd, dyd, 0.05)
    grad64 = sum(lo.rms_norm_backward(g64[m].reshape(T, n), xd, wd, rstd64)[0] for m in ("dq", "dk", "dv"))
    want64 = (grad64 * _np(real)).sum()
    truncation = abs(loss64(_np(up)) - loss64(_np(down)) - want64)
    c = ((192 + T) + 3 * (n / 16 + 24)) * 2.0 ** -24
    size = sum((np.abs(forward64(_np(x), lo.lin_forward_abs)[2]) * np.abs(dyd)).sum() for x in (up, down))
    gA = lo.lin_backward_abs(a64, a64, a64, ldd, dyd, 0.05)
    own = sum((2 * c * np.abs(wd) * np.abs(rstd64[:, None]) * gA[m].reshape(T, n) * (np.abs(_np(real)) + np.abs(_np(real)).mean())).sum()
              for m in ("dq", "dk", "dv"))
    bound = truncation + c * size + own
    assert abs(diff - want) <= bound
    assert abs(want) > 20 * bound
    for m, part in dx.items():  # without one of the parts
        assert abs(diff - want + (part * real).sum().item()) > 2 * bound, m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("operand,grad", [("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")])
def test_attention_along_the_gradient(cuda_ok, dtype, operand, grad):
    """The loss <y, dy> + <S_T, dS_T> is linear in each operand, so a difference of any length is
    exact but for rounding: sum |dy| tol(y) + sum |dS_T| tol(S_T) at both ends, and the gradient's
    own. The operand moves 64 times its size along the gradient, and all inputs are positive, so
    that the terms add up."""
    T, H, D = 200, 2, 64
    r = np.random.default_rng(3)
    unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True))
    s = {"q": unit(r.normal(size=(1, T, H, D))), "k": unit(r.normal(size=(1, T, H, D))), "v": r.normal(size=(1, T, H, D)),
         "dy": r.normal(size=(1, T, H, D)), "S0": r.normal(size=(1, H, D, D)), "dS_T": r.normal(size=(1, H, D, D))}
    t = {m: torch.tensor(np.abs(x), dtype=torch.float32).to(torch.float32 if m in ("S0", "dS_T") else dtype).cuda() for m, x in s.items()}
    ld = torch.tensor([-0.003, -0.2]).cuda()
    d, ldd = {m: _np(x) for m, x in t.items()}, _np(ld)
    g = muir.lin_attn_bwd(t["q"], t["k"], t["v"], ld, t["dy"], S0=t["S0"], dS_T=t["dS_T"])
    gA = lo.lin_backward_abs(d["q"], d["k"], d["v"], ldd, d["dy"], 1.0, None, d["S0"], d["dS_T"])

    def loss(x):
        y, S = muir.lin_attn_fwd(x["q"], x["k"], x["v"], ld, S0=x["S0"])
        yA, SA = lo.lin_forward_abs(*(_np(x[m]) for m in "qkv"), ldd, 1.0, None, _np(x["S0"]))
        slack = (d["dy"] * _tol(dtype, yA, yA, T, True)).sum() + (d["dS_T"] * _tol(dtype, SA, SA, T, False)).sum()
        return (y.double() * t["dy"].double()).sum().item() + (S.double() * t["dS_T"].double()).sum().item(), slack
    step = g[grad].double()
    step = step * (64 * t[operand].double().square().mean().sqrt() / step.square().mean().sqrt())
    moved = dict(t, **{operand: (t[operand].double() + step).to(t[operand].dtype)})
    real = moved[operand].double() - t[operand].double()
    (l1, s1), (l0, s0) = loss(moved), loss(t)
    want = (g[grad].double() * real).sum().item()
    bound = s1 + s0 + (np.abs(_np(real)) * _tol(dtype, gA[grad], gA[grad], T, operand != "S0")).sum()
    assert abs(l1 - l0 - want) <= bound
    assert want > 20 * bound


def test_every_round_of_two_calls_at_once(cuda_ok):
    """Calls on two streams, interleaved: each round of each as it is alone."""
    def work(seed, stream):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q, k, v, dy = (torch.randn(2, 900, 3, 64, generator=g, device="cuda").bfloat16() for _ in range(4))
        ld = -torch.rand(3, generator=g, device="cuda")
        x, w = torch.randn(64, 512, generator=g, device="cuda"), torch.randn(512, generator=g, device="cuda")
        codes = torch.randint(0, 16, (300, 512), generator=g, device="cuda", dtype=torch.uint8)
        packed = muir.w4_pack(codes, torch.rand(300, 8, generator=g, device="cuda").bfloat16())
        torch.cuda.synchronize()

        def call():
            y, S = muir.lin_attn_fwd(q, k, v, ld, stream=stream)
            gr = muir.lin_attn_bwd(q, k, v, ld, dy, stream=stream)
            f = muir.rms_norm(x, w, stream=stream)
            dx, dw = muir.rms_norm_bwd(x, x, w, f["rstd"], stream=stream)
            return [y, S, *gr.values(), f["y"], dx, dw, muir.w4_matvec(f["y"], *packed, 300, stream=stream)]
        return call
    calls = [work(i, torch.cuda.Stream()) for i in range(2)]
    alone = []
    for c in calls:
        alone.append(c())
        torch.cuda.synchronize()
    rounds = [[c() for c in calls] for _ in range(5)]
    torch.cuda.synchronize()
    for both in rounds:
        for a, b in zip(alone, both):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert muir.device_status() == 0
