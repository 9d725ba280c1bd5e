"""The layer operators together, as a layer uses them: a padded batch of prompts through
norm, projections and chunked attention, then tokens one by one through the norm's 8-bit
output, 4-bit projections and the recurrent step, against the same layer in 64 bits; and
a training step's gradients through norm and attention."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

B, T, H, D, DM = 3, 150, 2, 64, 256


def _weights():
    r = np.random.default_rng(0)
    W = {n: torch.tensor(r.normal(size=(H * D, DM)) / np.sqrt(DM), dtype=torch.float32).bfloat16().cuda() for n in "qkv"}
    packed, real = {}, {}
    for n, w in W.items():
        codes, scales = muir.w4_quantize(w, group=64)
        packed[n] = muir.w4_pack(codes, scales)
        real[n] = lo.w4_dequantize(codes.cpu().numpy(), scales.double().cpu().numpy())
    return packed, real, 1 + 0.1 * r.normal(size=DM), r


def test_prompt_then_tokens(cuda_ok):
    packed, real, wn, r = _weights()
    w = torch.tensor(wn, dtype=torch.float32).cuda()
    ld = torch.tensor([-0.01, -0.3]).cuda()
    lengths = [150, 77, 1]
    L = torch.tensor(lengths, dtype=torch.int32).cuda()
    x = torch.tensor(r.normal(size=(B, T, DM)), dtype=torch.float32).bfloat16().cuda()
    for b, n in enumerate(lengths):
        x[b, n:] = float("nan")  # padding holds anything
    f = muir.rms_norm(x.view(B * T, DM), w)
    q, k, v = (muir.w4_matvec(f["y"], *packed[n], H * D).view(B, T, H, D) for n in "qkv")
    y, S = muir.lin_attn_fwd(q, k, v, ld, scale=0.1, lengths=L)
    # each operator against 64 bits from what it was given: tolerances as in its own test file
    xd = x.double().cpu().numpy()
    for b, n in enumerate(lengths):
        yn, _, _ = lo.rms_norm(xd[b, :n], w.double().cpu().numpy())
        got = f["y"].view(B, T, DM)[b, :n].double().cpu().numpy()
        assert (np.abs(got - yn) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(yn)).all()
        qr = got @ real["q"].T
        assert (np.abs(q[b, :n].reshape(n, -1).double().cpu().numpy() - qr)
                <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -15 * (np.abs(got) @ np.abs(real["q"]).T)).all()
        a = [t[b:b + 1, :n].double().cpu().numpy() for t in (q, k, v)]
        yr, Sr = lo.lin_forward(*a, ld.double().cpu().numpy(), 0.1)
        yA, SA = lo.lin_forward_abs(*a, ld.double().cpu().numpy(), 0.1)
        assert (np.abs(y[b:b + 1, :n].double().cpu().numpy() - yr) <= 2.0 ** -8 * (np.abs(yr) + 1.02 * yA) + 2.0 ** -15 * yA).all()
        assert (np.abs(S[b].double().cpu().numpy() - Sr[0]) <= 2.0 ** -15 * SA[0]).all()
        assert (y[b, n:] == 0).all()
    # tokens, in 8 bits
    Sd = S.double().cpu().numpy()
    SA = np.abs(Sd)
    lam = np.exp(ld.double().cpu().numpy())[:, None, None]
    h = torch.zeros(B, DM, dtype=torch.bfloat16, device="cuda")
    for step in range(3):
        x1 = torch.tensor(r.normal(size=(B, DM)), dtype=torch.float32).bfloat16().cuda()
        o = muir.rms_norm_quant(x1, w, residual=h, h=h)
        t = {n: muir.w4_matvec(o["q"], *packed[n], H * D, x_scale=o["scale"]).view(B, H, D) for n in "qkv"}
        y1 = muir.lin_attn_step(S, t["q"], t["k"], t["v"], ld, scale=0.1)
        td = {n: a.double().cpu().numpy() for n, a in t.items()}
        xs = o["q"].double().cpu().numpy() * o["scale"].double().cpu().numpy()[:, None]
        vr = xs @ real["v"].T
        assert (np.abs(td["v"].reshape(B, -1) - vr) <= 2.0 ** -8 * np.abs(vr) + 2.0 ** -15 * (np.abs(xs) @ np.abs(real["v"]).T)).all()
        Sd = lam * Sd + td["k"][..., None] * td["v"][..., None, :]
        SA = lam * SA + np.abs(td["k"][..., None] * td["v"][..., None, :])
        yr = 0.1 * np.einsum("nhi,nhij->nhj", td["q"], Sd)
        yA = 0.1 * np.einsum("nhi,nhij->nhj", np.abs(td["q"]), SA)
        assert (np.abs(y1.double().cpu().numpy() - yr) <= 2.0 ** -8 * np.abs(yr) + 2.0 ** -14 * yA).all()
    assert (np.abs(S.double().cpu().numpy() - Sd) <= 2.0 ** -14 * SA).all()
    assert muir.device_status() == 0


def test_training_gradients_chain(cuda_ok):
    """d loss / d x through attention over the norm's output, fp32, against central
    differences of the whole chain. loss = <y, dy>, cubic in x's direction at most through
    q, k, v and smooth through the norm: a step of 2^-6 of a unit direction leaves
    step^2 / 6 of the third derivative, bounded here by 64 loss sizes, and the fp32
    rounding of the two losses, 2^-18 of the sum of absolute terms over the step."""
    r = np.random.default_rng(1)
    n = H * 32
    x = torch.tensor(r.normal(size=(1, 70, n)), dtype=torch.float32).cuda()
    w = torch.tensor(1 + 0.1 * r.normal(size=n), dtype=torch.float32).cuda()
    ld = torch.tensor([-0.02, -0.5]).cuda()
    dy = torch.tensor(r.normal(size=(1, 70, H, 32)), dtype=torch.float32).cuda()

    def forward(x):
        f = muir.rms_norm(x.view(70, n), w)
        a = f["y"].view(1, 70, H, 32)
        y, _ = muir.lin_attn_fwd(a, a, a, ld, scale=0.05)
        return f, a, y
    f, a, y = forward(x)
    g = muir.lin_attn_bwd(a, a, a, ld, dy, scale=0.05, want_dS0=False)
    da = (g["dq"].double() + g["dk"].double() + g["dv"].double()).float().view(70, n)
    dx, _ = muir.rms_norm_bwd(da, x.view(70, n), w, f["rstd"])
    e = torch.tensor(r.normal(size=(1, 70, n)), dtype=torch.float32).cuda()
    e = e / e.norm()
    step = 2.0 ** -6
    up, down = x + step * e, x - step * e
    loss = lambda x: (forward(x)[2].double() * dy.double()).sum().item()
    real = (up.double() - down.double()) / (2 * step)
    diff = (loss(up) - loss(down)) / (2 * step)
    size = (y.double().abs() * dy.double().abs()).sum().item()
    assert abs(diff - (dx.double().view_as(real) * real).sum().item()) <= 64 * size * step ** 2 / 6 + 2.0 ** -18 * size / step


def test_two_calls_at_once(cuda_ok):
    """Calls on two streams, interleaved: each as it is alone."""
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
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [work(i, s) for i, s in enumerate(streams)]
    alone = []
    for c in calls:
        alone.append(c())
        torch.cuda.synchronize()
    for _ in range(5):
        both = [c() for c in calls]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert muir.device_status() == 0
