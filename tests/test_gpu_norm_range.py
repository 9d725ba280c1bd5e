"""RMS norm of rows at the ends of fp32's range."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

pytestmark = pytest.mark.gpu


def _make(n, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = torch.tensor(r.normal(size=(n, d)), dtype=torch.float32).to(dtype).cuda()
    w = torch.tensor(1 + 0.2 * r.normal(size=d), dtype=torch.float32).cuda()
    return x, w


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
