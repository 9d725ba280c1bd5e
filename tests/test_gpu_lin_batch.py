"""A short sequence's result does not depend on what else is in its batch: a sequence of
one run of tokens gives the same bits alone, in a batch and padded."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,dk,dv", [(16, 64, 64), (4, 128, 128), (3, 32, 128)])
def test_alone_and_among_others(cuda_ok, dtype, H, dk, dv):
    B, T = 64, 48
    n = [1, 2, 5, 15, 16, 17, 31, 48]  # each at eight places of the batch
    lengths = torch.tensor(n * (B // len(n)), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k, v, dy = (make(B, T, H, d).to(dtype) for d in (dk, dk, dv, dv))
    S0, dS = make(B, H, dk, dv), make(B, H, dk, dv)
    ld = -torch.rand(H, generator=g, device="cuda")
    y, S = muir.lin_attn_fwd(q, k, v, ld, scale=0.1, lengths=lengths, S0=S0)
    gr = muir.lin_attn_bwd(q, k, v, ld, dy, scale=0.1, lengths=lengths, S0=S0, dS_T=dS)
    for b in [*range(8), B - 8, B - 1]:
        L = n[b % 8]
        a = [x[b:b + 1, :L].contiguous() for x in (q, k, v)]
        y1, S1 = muir.lin_attn_fwd(*a, ld, scale=0.1, S0=S0[b:b + 1])
        g1 = muir.lin_attn_bwd(*a, ld, dy[b:b + 1, :L].contiguous(), scale=0.1, S0=S0[b:b + 1], dS_T=dS[b:b + 1])
        assert torch.equal(y1[0], y[b, :L]) and torch.equal(S1[0], S[b]), L
        for m in ("dq", "dk", "dv"):
            assert torch.equal(g1[m][0], gr[m][b, :L]), (m, L)
        assert torch.equal(g1["dS0"][0], gr["dS0"][b]), L
    assert muir.device_status() == 0
