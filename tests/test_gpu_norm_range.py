"""RMS norm of rows at the ends of fp32's range: rows of zeros without an epsilon, rows
whose squares underflow, rows whose squares overflow. Tolerances as in the norm's other
tests: the sum of squares errs by (d / 8 + 16) 2^-24 of itself, rstd by half of that."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _make(n, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = torch.tensor(r.normal(size=(n, d)), dtype=torch.float32).to(dtype).cuda()
    w = torch.tensor(1 + 0.2 * r.normal(size=d), dtype=torch.float32).cuda()
    return x, w


def _np(x):
    return x.double().cpu().numpy()


DIMS = [8, 256, 264, 1000, 2048, 4104, 16384]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("residual", [False, True])
def test_rows_of_zeros_without_an_epsilon(cuda_ok, dtype, dim, residual):
    x, w = _make(3, dim, dtype, 0)
    x[1] = 0.0
    res = torch.zeros_like(x) if residual else None
    o = muir.rms_norm(x, w, residual=res, eps=0.0)
    q = muir.rms_norm_quant(x, w, residual=res, eps=0.0)
    assert (o["y"][1] == 0).all() and o["rstd"][1] == 0
    assert (q["q"][1].float() == 0).all() and q["scale"][1] == 0 and q["rstd"][1] == 0
    for i in (0, 2):
        alone = muir.rms_norm(x[i:i + 1].contiguous(), w, residual=None if res is None else res[:1], eps=0.0)
        assert torch.equal(o["y"][i:i + 1], alone["y"]) and o["y"][i].isfinite().all()
    dy, _ = _make(3, dim, dtype, 1)
    dx, dw = muir.rms_norm_bwd(dy, x, w, o["rstd"], dh=dy)
    assert torch.equal(dx[1], dy[1]) and dx.isfinite().all() and dw.isfinite().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("size,eps", [(2.0 ** -84, 0.0), (2.0 ** -66, 0.0), (2.0 ** -84, 2.0 ** -166), (2.0 ** -84, 2.0 ** -140),
                                      (2.0 ** 65, 1e-6), (2.0 ** 83, 1e-6), (2.0 ** 120, 0.0)])
def test_rows_whose_squares_leave_the_range(cuda_ok, dtype, dim, size, eps):
    eps = float(np.float32(eps))  # 2^-166 is 0 in the operator's fp32
    x, w = _make(4, dim, dtype, 2)
    x = (x.float() * size).to(dtype)
    x[2] = (x[2].float() / size).to(dtype)  # an ordinary row among them
    x[3, 1:] = 0.0  # one element that is far above the others
    xd, wd = _np(x), _np(w)
    y, _, rstd = lo.rms_norm(xd, wd, eps=eps)
    c = (dim / 16 + 26) * U
    o = muir.rms_norm(x, w, eps=eps)
    assert (np.abs(_np(o["rstd"]) - rstd) <= c * rstd).all()
    assert (np.abs(_np(o["y"]) - y) <= (c + HALF[dtype]) * np.abs(y) + 1e-38).all()
    q = muir.rms_norm_quant(x, w, eps=eps)
    assert torch.equal(q["rstd"], o["rstd"])
    scale = np.abs(y).max(-1) / 448.0
    assert (np.abs(_np(q["scale"]) - scale) <= 2 * c * scale).all()
    z, got = y / scale[:, None], _np(q["q"])
    near = np.minimum(np.abs(got - lo.e4m3(z * (1 + 4 * c))), np.abs(got - lo.e4m3(z * (1 - 4 * c))))
    assert (near == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_and_nan_are_not_taken_for_large_rows(cuda_ok, dtype):
    x, w = _make(5, 2048, dtype, 3)
    x *= 2.0 ** 80
    x[0, 5] = float("inf")
    x[1, 6] = float("nan")
    x[2, 7], x[2, 9] = float("inf"), float("nan")
    x[3, 11] = -float("inf")
    o = muir.rms_norm(x, w)
    for i in (0, 3):
        assert o["rstd"][i] == 0 and o["y"][i].isnan().sum() == 1 and (o["y"][i][~o["y"][i].isnan()] == 0).all()
    assert o["y"][1].isnan().all() and o["y"][2].isnan().all()
    assert o["y"][4].isfinite().all() and o["y"][4].abs().max() > 1


def test_subnormal_rows(cuda_ok):
    """1 / rms of a subnormal row is above fp32's largest number, its norm is not."""
    x = torch.tensor([[1.0, -2.0, 3.0, 0.0, 5.0, 1.0, 0.0, 1.0]]).cuda() * 2.0 ** -140
    w = torch.ones(8).cuda()
    o = muir.rms_norm(x, w, eps=0.0)
    y, _, _ = lo.rms_norm(_np(x), _np(w), eps=0.0)
    assert (np.abs(_np(o["y"]) - y) <= 32 * U * np.abs(y)).all()
    assert o["rstd"].item() == float("inf")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [2048, 4104, 16384])
def test_rows_with_infinities_in_8_bits_again_and_again(cuda_ok, dtype, dim):
    """Every other row holds an infinity: no row of any call differs from the first call's."""
    x, w = _make(64, dim, dtype, 4)
    x[::2, dim // 3] = float("inf")
    first = muir.rms_norm_quant(x, w)
    assert first["scale"][::2].isnan().all() and first["scale"][1::2].isfinite().all() and (first["rstd"][::2] == 0).all()
    bits = {m: first[m].view(torch.uint8) for m in first}
    differing = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        o = muir.rms_norm_quant(x, w)
        differing += sum((o[m].view(torch.uint8) != bits[m]).sum() for m in bits)
    assert differing.item() == 0
