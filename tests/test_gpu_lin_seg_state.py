"""The states that segments hand on are fp32 sums of exact products, whether a final state
is wanted or not.

The first segment's tokens write positive values and its last three cancel them, so that
the state handed on is zero up to its own rounding; the first token behind it reads that
state and nothing else. Keys are the same at every token, so one value per column cancels
all rows. With a decay of 2^(-1/16) the last 16 tokens hold half of the sum A of absolute
terms, the 16 before them a quarter: the tensor core's accumulator, which cuts after each
step of 16 tokens, loses at most 2^-23 (A/2 + A/4 + ..) = 2^-23 A, fp32 products of a key
and its weight 2^-24 A, and weights of their own 2 x 2^-24 A each: 8 x 2^-24 A with the
carry and the read, and as much again for steps whose parts cut more than once."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from tests.test_gpu_lin_segments import _segments

pytestmark = pytest.mark.gpu
T, D = 4096, 64


@pytest.mark.parametrize("backward", [False, True])
def test_the_state_handed_on_is_exact(cuda_ok, backward):
    r = np.random.default_rng(0)
    bf = lambda x: torch.tensor(x, dtype=torch.float32).bfloat16().double().numpy()
    ld = torch.tensor([-math.log(2.0) / 16])
    lam = math.exp(ld.double().item())
    z = torch.zeros(1, T, 1, D, dtype=torch.bfloat16, device="cuda")
    n, chunks = _segments({"q": z, "k": z, "v": z, "ld": ld.cuda()}, backward)
    assert n > 1
    L = 128 * chunks  # the first segment
    key, v = bf(1 + r.random(D)), np.zeros((L, D))
    w = lam ** np.arange(L - 1, -1, -1.0)
    v[:L - 3] = bf(0.5 + r.random((L - 3, D)))
    for t in (L - 1, L - 2, L - 3):  # the weights 1, lambda, lambda^2: -sum, then what its rounding left
        v[t] = bf(-(w @ v) / w[t])
    # read with ones over the other dimension: y over rows, dq over columns
    S, A = np.outer(key, w @ v), np.outer(key, w @ np.abs(v))
    ref, A = lam * S.sum(1 if backward else 0), lam * A.sum(1 if backward else 0)
    k, vv, one = z.clone(), z.clone(), z.clone()
    k[0, :L, 0] = torch.tensor(key)
    vv[0, :L, 0] = torch.tensor(v)
    one[0, L] = 1.0
    if backward:
        got = muir.lin_attn_bwd(z, k, vv, ld.cuda(), one)["dq"]
    else:
        got = muir.lin_attn_fwd(one, k, vv, ld.cuda(), want_state=False)[0]
    err = np.abs(got[0, L, 0].double().cpu().numpy() - ref)
    tol = 16 * 2.0 ** -24 * A + 2.0 ** -7 * np.abs(ref)
    assert (np.abs(ref) < 2.0 ** -22 * A).all()  # it does cancel
    assert (err <= tol).all(), f"{(err / tol).max():.3g} times the bound"
