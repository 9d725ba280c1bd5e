"""Padded batches again and again: whatever the order in which the tiles of a chunk arrive,
padding (NaN here) reaches no output, and every call gives the bits of the first. The
sequences end inside their second, third and fifth chunk, in one segment, with one sequence
and head per SM and with more."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(36, 307, 4, 128, 128), (33, 588, 4, 128, 32), (24, 520, 6, 64, 128), (80, 300, 4, 128, 64)])
@pytest.mark.parametrize("state", [False, True])
def test_padding_never_arrives(cuda_ok, case, state):
    B, T, H, dk, dv = case
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, dy = (torch.randn(B, T, H, d, generator=g, device="cuda").bfloat16() for d in (dk, dk, dv, dv))
    L = torch.randint(129, T, (B,), generator=g, device="cuda", dtype=torch.int32)
    L[::3] = T
    live = torch.arange(T, device="cuda")[None] < L[:, None]
    for x in (q, k, v, dy):
        x[~live] = float("nan")
    ld = torch.tensor([-1e-4, -2.7, -0.01, 0.0, -0.3, -0.1][:H], device="cuda")

    def call():
        y, S = muir.lin_attn_fwd(q, k, v, ld, lengths=L, want_state=state)
        gr = muir.lin_attn_bwd(q, k, v, ld, dy, lengths=L, want_dS0=state)
        return [x for x in (y, S, *gr.values()) if x is not None]
    first = call()
    assert all(x.isfinite().all() for x in first) and all((x[~live] == 0).all() for x in first if x.ndim == 4 and x.shape[:2] == (B, T))
    differing = torch.zeros(len(first), dtype=torch.int64, device="cuda")
    for _ in range(400):
        differing += torch.stack([(a != b).any() for a, b in zip(call(), first)])
    assert differing.tolist() == [0] * len(first)
    assert muir.device_status() == 0
