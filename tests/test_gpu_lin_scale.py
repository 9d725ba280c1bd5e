"""Scales that make large weights of small products (tolerances as in the operator's other tests)."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo
from tests.test_gpu_lin_attn import _check, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("power", [40, 59, 61, 90, 110])
@pytest.mark.parametrize("T", [5, 300])
def test_scales_far_above_one(cuda_ok, dtype, power, T):
    """q is small by the same power of two as the scale is large, so outputs are ordinary numbers."""
    ld = [-2.6, -2.7, -2.8, -0.001, -30.0]
    d, t = _make(1, T, len(ld), 64, 64, dtype, seed=30, log_decay=ld)
    up = 2.0 ** power
    t["q"], d["q"] = (t["q"].float() / up).to(dtype), d["q"] / up
    y, S = muir.lin_attn_fwd(t["q"], t["k"], t["v"], t["ld"], scale=up, S0=t["S0"])
    a = (d["q"], d["k"], d["v"], d["ld"], up, None, d["S0"])
    _check("y", y, lo.lin_forward(*a)[0], lo.lin_forward_abs(*a)[0], T, dtype)
    g = muir.lin_attn_bwd(t["q"], t["k"], t["v"], t["ld"], t["dy"], scale=up, S0=t["S0"], dS_T=t["dS_T"])
    b = (d["q"], d["k"], d["v"], d["ld"], d["dy"], up, None, d["S0"], d["dS_T"])
    gr, gA = lo.lin_backward(*b), lo.lin_backward_abs(*b)
    for n, by in (("dk", 1.0), ("dv", 1.0), ("dq", up)):  # dq is as large as the scale
        _check(n, g[n] / by, gr[n] / by, gA[n] / by, T, dtype)
    _check("dS0", g["dS0"], gr["dS0"], gA["dS0"], T, dtype, out=False)
    assert muir.device_status() == 0
