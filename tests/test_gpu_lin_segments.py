"""Linear attention over segments of several chunks each: the segment states, their
combination and the outputs from them, forward and backward, against the 64-bit
recurrence of two of the heads. Tolerances as in the operator's other tests."""
import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from oracle import layer_oracle as lo
from tests.test_gpu_lin_attn import _check, _make

pytestmark = pytest.mark.gpu
CHUNK = 128


def _segments(t, backward):
    """(segments, chunks in each), from the workspace that the split needs."""
    B, T, H, dk = t["q"].shape
    state = B * H * dk * t["v"].shape[-1] * 4
    n = muir.lin_attn_workspace_bytes(t["q"], t["k"], t["v"], t["ld"], backward=backward) // (state * (2 if backward else 1))
    return n, -(-(-(-T // CHUNK)) // n) if n else 1


def _slow(H):
    """Decays by which the first tokens still count at the end, for the first and the last head; faster ones between."""
    return [-1e-4] + [-0.02] * (H - 2) + [-7e-4]


@pytest.mark.parametrize("case", [(1, 4000, 8, 128, 128), (1, 4000, 8, 64, 128), (1, 4000, 8, 128, 64), (2, 2900, 4, 64, 64),
                                  (2, 2900, 4, 32, 128), (2, 2900, 4, 128, 32)])
@pytest.mark.parametrize("lengths", ["full", "ragged"])
@pytest.mark.parametrize("state", [False, True])
def test_segments_of_several_chunks(cuda_ok, case, lengths, state):
    B, T, H, dk, dv = case
    d, t = _make(*case, torch.bfloat16, seed=20, log_decay=_slow(H))
    for backward in (False, True):
        n, chunks = _segments(t, backward)
        assert n > 1 and chunks > 1  # or the case does not test what it says
    # ragged: the last sequence ends inside a chunk of its second segment, so that later segments hold no token
    L = None if lengths == "full" else [T] * (B - 1) + [CHUNK * chunks + 131]
    Lt = None if L is None else torch.tensor(L, dtype=torch.int32, device="cuda")
    if L is not None:
        for x in ("q", "k", "v", "dy"):
            t[x][B - 1, L[-1]:] = float("nan")
            d[x][B - 1, L[-1]:] = 0.0
    S0, dS = ("S0", "dS_T") if state else (None, None)
    a = (t["q"], t["k"], t["v"], t["ld"])
    kw = dict(scale=0.125, lengths=Lt, S0=t.get(S0))
    y, S = muir.lin_attn_fwd(*a, **kw)
    y2, _ = muir.lin_attn_fwd(*a, want_state=False, **kw)
    g = muir.lin_attn_bwd(*a, t["dy"], dS_T=t.get(dS), **kw)
    g2 = muir.lin_attn_bwd(*a, t["dy"], dS_T=t.get(dS), want_dS0=False, **kw)
    h = [0, H - 1]
    o = (d["q"][:, :, h], d["k"][:, :, h], d["v"][:, :, h], d["ld"][h])
    s0, dsT = (d["S0"][:, h], d["dS_T"][:, h]) if state else (None, None)
    yr, Sr = lo.lin_forward(*o, 0.125, L, s0)
    yA, SA = lo.lin_forward_abs(*o, 0.125, L, s0)
    gr = lo.lin_backward(*o, d["dy"][:, :, h], 0.125, L, s0, dsT)
    gA = lo.lin_backward_abs(*o, d["dy"][:, :, h], 0.125, L, s0, dsT)
    for got in (y, y2):
        _check("y", got[:, :, h], yr, yA, T, torch.bfloat16)
    _check("S_T", S[:, h], Sr, SA, T, torch.bfloat16, out=False)
    for n in ("dq", "dk", "dv"):
        for got in (g, g2):
            _check(n, got[n][:, :, h], gr[n], gA[n], T, torch.bfloat16)
    _check("dS0", g["dS0"][:, h], gr["dS0"], gA["dS0"], T, torch.bfloat16, out=False)
    if L is not None:
        for x in (y, g["dq"], g["dk"], g["dv"]):
            assert (x[B - 1, L[-1]:] == 0).all()
    assert muir.device_status() == 0
