"""RMS norm with the residual's addition against its formula in 64 bits.

Tolerances, elementwise. The sum of d squares errs by at most (d / 8 + 16) 2^-24 of
itself (8 chains per thread, then a tree), which rstd halves; with the root, the
division and the two products y is within (d / 16 + 24) 2^-24 |y| and one rounding of
its type: 2^-8 |y| for bf16. Outputs in 8 bits are exact but for values within that
distance of the middle between two codes, which may go to either."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _make(n, d, dtype, seed=0):
    r = np.random.default_rng(seed)
    t = {m: torch.tensor(r.normal(size=(n, d)), dtype=torch.float32).to(dtype).cuda() for m in ("x", "res", "dy", "dh")}
    t["w"] = torch.tensor(1 + 0.2 * r.normal(size=d), dtype=torch.float32).cuda()
    return {m: x.double().cpu().numpy() for m, x in t.items()}, t


def _close(name, got, ref, tol):
    got = got.double().cpu().numpy()
    bad = np.abs(got - ref) > tol + 1e-30
    assert not bad.any(), f"{name}: {np.abs(got - ref)[bad].max():.3g} off at {np.argwhere(bad)[0]}"


SIZES = [(1, 8), (3, 40), (17, 256), (5, 264), (33, 512), (9, 1000), (2, 1024), (7, 1032), (40, 2048), (3, 4096),
         (2, 5000), (1, 8192), (2, 8200), (1, 16384)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(cuda_ok, dtype, size, residual):
    n, dim = size
    d, t = _make(n, dim, dtype)
    kw = dict(residual=t["res"] if residual else None, eps=1e-5)
    o = muir.rms_norm(t["x"], t["w"], **kw)
    y, h, rstd = lo.rms_norm(d["x"], d["w"], d["res"] if residual else None, 1e-5)
    c = (dim / 16 + 24) * U
    _close("rstd", o["rstd"], rstd, c * rstd)
    _close("y", o["y"], y, (c + HALF[dtype]) * np.abs(y))
    assert ("h" in o) == residual
    if residual:
        _close("h", o["h"], h, (HALF[dtype] + U) * np.abs(h))
    q = muir.rms_norm_quant(t["x"], t["w"], **kw)
    assert torch.equal(q["rstd"], o["rstd"]) and (not residual or torch.equal(q["h"], o["h"]))
    scale = np.abs(y).max(-1) / 448.0
    _close("scale", q["scale"], scale, 2 * c * scale)
    z = y / scale[:, None]
    got = q["q"].double().cpu().numpy()
    near = np.minimum(np.abs(got - lo.e4m3(z * (1 + 4 * c))), np.abs(got - lo.e4m3(z * (1 - 4 * c))))
    assert (near == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES + [(700, 2048), (1300, 24)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(cuda_ok, dtype, size, residual):
    n, dim = size
    d, t = _make(n, dim, dtype, seed=1)
    o = muir.rms_norm(t["x"], t["w"])
    rstd = o["rstd"].double().cpu().numpy()
    dx, dw = muir.rms_norm_bwd(t["dy"], t["x"], t["w"], o["rstd"], dh=t["dh"] if residual else None)
    rx, rw = lo.rms_norm_backward(d["dy"], d["x"], d["w"], rstd, d["dh"] if residual else None)
    g, xh = np.abs(d["dy"] * d["w"]), np.abs(d["x"] * rstd[:, None])
    A = rstd[:, None] * (g + xh * np.mean(g * xh, -1, keepdims=True)) + (np.abs(d["dh"]) if residual else 0.0)
    _close("dx", dx, rx, (dim / 8 + 24) * U * A + HALF[dtype] * np.abs(rx))
    _close("dweight", dw, rw, (n + 4) * U * np.sum(np.abs(d["dy"]) * xh, 0))
    again = muir.rms_norm_bwd(t["dy"], t["x"], t["w"], o["rstd"], dh=t["dh"] if residual else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_against_differences(cuda_ok):
    """Central differences of the fp32 forward: step h = 2^-7 leaves h^2 / 6 of the third
    derivative (below 8 per element sum) and 2^-24 of the loss over 2 h."""
    d, t = _make(4, 64, torch.float32, seed=2)
    o = muir.rms_norm(t["x"], t["w"], residual=t["res"])
    dx, dw = muir.rms_norm_bwd(t["dy"], o["h"], t["w"], o["rstd"], dh=t["dh"])

    def loss(x, w):
        f = muir.rms_norm(x, w, residual=t["res"])
        return ((f["y"].double() * t["dy"].double()).sum() + (f["h"].double() * t["dh"].double()).sum()).item()
    step, r = 2.0 ** -7, torch.Generator().manual_seed(0)
    for grad, x, at in ((dx, t["x"], 0), (dw, t["w"], 1)):
        e = torch.randn(x.shape, generator=r).cuda()
        args = [t["x"], t["w"]]
        up, down = list(args), list(args)
        up[at], down[at] = x + step * e, x - step * e
        real = (up[at].double() - down[at].double()) / (2 * step)
        diff = (loss(*up) - loss(*down)) / (2 * step)
        size = (real.abs() * grad.abs().double()).sum().item()
        assert abs(diff - (grad.double() * real).sum().item()) <= 8 * step ** 2 / 6 * real.abs().sum().item() + 2.0 ** -24 / step * 4 * size


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_zeros_infinities_and_nan(cuda_ok, dtype):
    d, t = _make(6, 1040, dtype, seed=3)
    x = t["x"]
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 1e-30 if dtype == torch.float32 else 2.0 ** -100
    q = muir.rms_norm_quant(x, t["w"], eps=0.0 if False else 1e-6)
    o = muir.rms_norm(x, t["w"])
    assert (q["q"][0].float() == 0).all() and q["scale"][0] == 0 and (o["y"][0] == 0).all()
    assert o["y"][1, 3].isnan() and (o["y"][1, 4:] == 0).all() and q["scale"][1].isnan()
    assert o["y"][2].isnan().all() and q["q"][2].float().isnan().all()
    # far below eps: y = x w / sqrt(eps); the codes still span e4m3's range
    assert q["q"][3].float().abs().max() == 448
    y3 = x[3].double() * t["w"].double() * 1e3
    err = (q["q"][3].double() * (y3.abs().max() / 448) - y3).abs()
    assert (err <= 2.0 ** -4 * 1.01 * y3.abs() + 2.0 ** -10 * 1.01 * y3.abs().max() / 448).all()
    # the other rows are what they are alone
    alone = muir.rms_norm(x[4:].contiguous(), t["w"])
    assert torch.equal(alone["y"], o["y"][4:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_empty_stream_and_graph(cuda_ok, dtype):
    d, t = _make(50, 2048, dtype, seed=4)
    want = muir.rms_norm(t["x"], t["w"], residual=t["res"])
    dwant = muir.rms_norm_bwd(t["dy"], want["h"], t["w"], want["rstd"], dh=t["dh"])
    x, res = t["x"].clone(), t["res"].clone()
    got = muir.rms_norm(x, t["w"], residual=res, y=x, h=res)
    assert torch.equal(x, want["y"]) and torch.equal(res, want["h"]) and got["h"] is res
    dy = t["dy"].clone()
    dx, dw = muir.rms_norm_bwd(dy, want["h"], t["w"], want["rstd"], dh=t["dh"], dx=dy)
    assert torch.equal(dx, dwant[0]) and torch.equal(dw, dwant[1])
    e = muir.rms_norm(t["x"][:0], t["w"], residual=t["res"][:0])
    assert e["y"].shape == (0, 2048) and e["rstd"].shape == (0,)
    dx, dw = muir.rms_norm_bwd(t["dy"][:0], e["h"], t["w"], e["rstd"])
    assert dx.shape == (0, 2048) and (dw == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = muir.rms_norm_bwd(t["dy"], want["h"], t["w"], want["rstd"], dh=t["dh"], stream=side)
    side.synchronize()
    assert torch.equal(s[0], dwant[0]) and torch.equal(s[1], dwant[1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        f = muir.rms_norm(t["x"], t["w"], residual=t["res"])
        b = muir.rms_norm_bwd(t["dy"], f["h"], t["w"], f["rstd"], dh=t["dh"])
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(f["y"], want["y"]) and torch.equal(b[0], dwant[0]) and torch.equal(b[1], dwant[1])


def test_offsets_past_32_bits(cuda_ok):
    n, dim = 140_000, 16384
    x = torch.zeros(n, dim, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(dim, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    w = torch.ones(dim, device="cuda")
    o = muir.rms_norm(x, w)
    y, _, _ = lo.rms_norm(x[-1:].double().cpu().numpy(), w.double().cpu().numpy())
    _close("y", o["y"][-1:], y, ((dim / 16 + 24) * U + 2.0 ** -8) * np.abs(y))
    assert (o["y"][-3:-1] == 0).all()
    dx, dw = muir.rms_norm_bwd(x, x, w, o["rstd"])
    rx, rw = lo.rms_norm_backward(x[-1:].double().cpu().numpy(), x[-1:].double().cpu().numpy(), 1.0,
                                  o["rstd"][-1:].double().cpu().numpy())
    _close("dweight", dw, rw, 8 * U * np.abs(rw))
