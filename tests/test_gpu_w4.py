"""Products with 4-bit weights against the dequantised product in 64 bits.

Tolerances, elementwise, with A = sum |x| |w|: fp32 sums over K terms err by at most
(K + 16) 2^-24 A, and a bf16 result is rounded once, 2^-8 |y|. Weights, bf16 and e4m3
rows are exact in the products; fp32 rows are three parts that sum to them exactly."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def _weights(O, K, group, seed=0):
    r = np.random.default_rng(seed)
    codes = torch.tensor(r.integers(0, 16, (O, K)), dtype=torch.uint8).cuda()
    scales = torch.tensor(r.uniform(0.1, 1.0, (O, K // group)) / np.sqrt(K), dtype=torch.float32).bfloat16().cuda()
    return codes, scales, lo.w4_dequantize(codes.cpu().numpy(), scales.double().cpu().numpy())


def _rows(n, K, kind, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, K, generator=g)
    if kind != "e4m3":
        x = x.to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()
        return x, None, x.double().cpu().numpy()
    s = x.abs().amax(-1) / 448.0
    q = (x / s[:, None]).to(E4M3)
    return q.cuda(), s.cuda(), q.double().numpy() * s.double().numpy()[:, None]


def _check(y, xd, W):
    ref, A = xd @ W.T, np.abs(xd) @ np.abs(W).T
    tol = (xd.shape[1] + 16) * 2.0 ** -24 * A + (2.0 ** -8 * np.abs(ref) if y.dtype == torch.bfloat16 else 0.0) + 1e-30
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.3g} times the bound"


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [(1, 16, 128), (1, 1, 256), (3, 17, 1152), (8, 100, 2048), (9, 33, 128), (16, 48, 384),
                                  (31, 65, 640), (33, 50, 256), (70, 16, 1024)])
def test_matvec(cuda_ok, kind, group, size):
    n, O, K = size
    codes, scales, W = _weights(O, K, group)
    wq, ws = muir.w4_pack(codes, scales)
    x, xs, xd = _rows(n, K, kind)
    y = muir.w4_matvec(x, wq, ws, O, x_scale=xs)
    assert y.shape == (n, O) and y.dtype == (torch.float32 if kind == "f32" else torch.bfloat16)
    _check(y, xd, W)
    if kind == "e4m3":
        _check(muir.w4_matvec(x, wq, ws, O, x_scale=xs, out_dtype=torch.float32), xd, W)
        _check(muir.w4_matvec(x, wq, ws, O), x.double().cpu().numpy(), W)
    # a row's result does not depend on the other rows
    assert torch.equal(muir.w4_matvec(x[:1].contiguous(), wq, ws, O, x_scale=None if xs is None else xs[:1].contiguous()), y[:1])


@pytest.mark.parametrize("size", [(16, 128, 128), (19, 256, 32), (40, 384, 64)])
def test_pack_writes_the_documented_layout(cuda_ok, size):
    O, K, group = size
    codes, scales, _ = _weights(O, K, group)
    wq, ws = muir.w4_pack(codes | 0xA0, scales)  # only the low four bits of a code count
    rq, rs = lo.w4_layout(codes.cpu().numpy(), scales.double().cpu().numpy())
    assert (wq.cpu().numpy() == rq).all() and (ws.double().cpu().numpy() == rs).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(cuda_ok, dtype, group):
    g = torch.Generator().manual_seed(2)
    w = torch.randn(37, 512, generator=g).to(dtype)
    w[3, :128] = 0.0
    codes, scales = muir.w4_quantize(w.cuda(), group=group)
    c, s, wd = codes.cpu().numpy().astype(np.int64), scales.double().cpu().numpy(), w.double().numpy()
    top = np.abs(wd.reshape(37, -1, group)).max(-1)
    assert (np.abs(s - top / 7) <= 2.0 ** -8 * top / 7 * (1 + 2.0 ** -14)).all()
    assert (c[3, :128] == 8).all() and c.min() >= 0 and c.max() <= 15
    sr = np.repeat(s, group, axis=1)
    err = np.abs((c - 8) * sr - wd)
    # half a step, but for weights that the bf16 scale puts past code 15 (7 scale < |w| <= 7 scale (1 + 2^-8))
    assert (err <= sr * (0.5 + 7 * 2.0 ** -8 * 1.01) + 1e-30).all()
    wq, ws = muir.w4_pack(codes, scales)
    x, _, xd = _rows(4, 512, "bf16")
    _check(muir.w4_matvec(x, wq, ws, 37), xd, lo.w4_dequantize(c, s))


def test_infinities_nan_and_large_values_stay_in_their_row(cuda_ok):
    codes, scales, W = _weights(40, 256, 64)
    codes[:] = codes.clamp(min=9)  # no zero weights: an infinity stays one
    W = lo.w4_dequantize(codes.cpu().numpy(), scales.double().cpu().numpy())
    wq, ws = muir.w4_pack(codes, scales)
    for kind in ("f32", "bf16"):
        x, _, _ = _rows(6, 256, kind)
        x[1, 7], x[2, 9] = float("inf"), float("nan")
        x[3, 0] = torch.finfo(torch.float32).max if kind == "f32" else 1e38
        y = muir.w4_matvec(x, wq, ws, 40)
        assert (y[1] == float("inf")).all() and y[2].isnan().all()
        keep = [0, 4, 5] if W.max() * 4e38 > 3.4e38 else [0, 3, 4, 5]
        xk = x[keep].contiguous()
        _check(y[keep], xk.double().cpu().numpy(), W)
        assert y[3].isfinite().all() == (np.abs(x[3].double().cpu().numpy() @ W.T).max() < 3.3e38)


def test_empty_stream_graph_and_large(cuda_ok):
    codes, scales, W = _weights(5000, 2048, 128)
    wq, ws = muir.w4_pack(codes, scales)
    x, _, xd = _rows(3, 2048, "bf16")
    assert muir.w4_matvec(x[:0], wq, ws, 5000).shape == (0, 5000)
    want = muir.w4_matvec(x, wq, ws, 5000)
    _check(want, xd, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = muir.w4_matvec(x, wq, ws, 5000, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = muir.w4_matvec(x, wq, ws, 5000)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_refusals_on_the_device(cuda_ok):
    codes, scales, _ = _weights(20, 256, 64)
    wq, ws = muir.w4_pack(codes, scales)
    x, xs, _ = _rows(2, 256, "e4m3")
    with pytest.raises(ValueError, match="inputs"):
        muir.w4_matvec(x[:, :128].contiguous(), wq, ws, 20)
    for O in (0, 16, 33):
        with pytest.raises(ValueError, match="outputs"):
            muir.w4_matvec(x, wq, ws, O)
    with pytest.raises(ValueError, match="x_scale"):
        muir.w4_matvec(x.bfloat16(), wq, ws, 20, x_scale=xs)
    with pytest.raises(TypeError, match="out_dtype"):
        muir.w4_matvec(x.bfloat16(), wq, ws, 20, out_dtype=torch.float32)
