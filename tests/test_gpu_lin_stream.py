"""Streams of single tokens decay like prompts.

A decay near 1 that is rounded to fp32 before it multiplies the state is off by the same
amount at every token: half of 2^-24 a token for the slowest decays here, which adds up
to the number of tokens times that. Rounding the state itself is different: those errors
change their sign from token to token. So the bound is that of a sum of independent errors.
Each token's roundings are at most c_t = 2^-24 S_t (the writes are positive, so S_t grows
to its final value and is its own sum of absolute values); after n tokens c_t has decayed
by lambda^(n-t), so the squares sum to at most (2^-24 S_n)^2 m with m = min(n, 1 / (2 |log
lambda|)); and a sum of independent errors exceeds 8 times the root of that with a
probability below 2 exp(-32) = 3e-14 (Hoeffding). 8 more roundings are for the last
token's sums and for the rounding of 1 - lambda, which is relative to 1 - lambda."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

pytestmark = pytest.mark.gpu
N = 40_000
# 1e-4; 1e-6; one and a half units of the last place below 1; exp(-0.8), where a state lives for few tokens
DECAYS = [-1e-4, -1e-6, -1.5 * 2.0 ** -24, -0.8]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dims", [(32, 32), (128, 64)])
def test_a_long_stream_keeps_its_decay(cuda_ok, dtype, dims):
    dk, dv = dims
    H = len(DECAYS)
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (0.5 + torch.rand(N, 1, H, d, generator=g, device="cuda") for d in dims)
    k, v = k.to(dtype), v.to(dtype)
    ld = torch.tensor(DECAYS, device="cuda")
    S = torch.zeros(1, H, dk, dv, device="cuda")
    y = None
    for i in range(N):
        y = muir.lin_attn_step(S, k[i], k[i], v[i], ld, scale=0.25, y=y)
    left = torch.arange(N - 1, -1, -1, device="cuda", dtype=torch.float64)
    w = torch.exp(ld.double()[None] * left[:, None])  # [N,H]
    kd, vd = k[:, 0].double(), v[:, 0].double()
    ref = torch.einsum("nh,nhi,nhj->hij", w, kd, vd)
    m = torch.clamp(1 / (2 * ld.double().abs()), max=N)
    tol = (8 * m.sqrt() + 8) * 2.0 ** -24
    over = ((S[0].double() - ref).abs() / ref).amax((1, 2)) / tol
    assert (over <= 1).all(), f"{over.tolist()} times the bound, by decay"
    yr = 0.25 * torch.einsum("hi,hij->hj", kd[-1], ref)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    # every term of y is positive: its state's bound, 128 roundings of the sum, one of the output
    assert ((y[0].double() - yr).abs() <= (tol[:, None] + 130 * 2.0 ** -24 + half * (1 + 2.0 ** -7)) * yr).all()
    assert muir.device_status() == 0
