"""Products with 4-bit weights of so many outputs that a CTA takes two tiles of 16: the
last size that takes one, the first that takes two, and an odd count of tiles with a
partial last one, whose second tile lies past the end. Tolerances as in the product's
other tests: (K + 16) 2^-24 of the sum of absolute terms, one rounding for bf16."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def _rows(n, K, kind, g):
    x = torch.randn(n, K, generator=g, device="cuda")
    if kind != "e4m3":
        x = x.to(torch.float32 if kind == "f32" else torch.bfloat16)
        return x, None, x.double()
    s = x.abs().amax(-1) / 448.0
    q = (x / s[:, None]).to(E4M3)
    return q, s, q.double() * s.double()[:, None]


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("O,K", [(37872, 128), (37873, 128), (37873, 640), (37889, 128), (37889, 640), (37904, 256)])
def test_two_tiles_per_block(cuda_ok, kind, group, O, K):
    g = torch.Generator(device="cuda").manual_seed(O + K)
    codes = torch.randint(0, 16, (O, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.1 + torch.rand(O, K // group, generator=g, device="cuda")) / K ** 0.5).bfloat16()
    packed = muir.w4_pack(codes, scales)
    W = (codes.double() - 8.0) * scales.double().repeat_interleave(group, 1)
    for n in (1, 8, 9, 16, 17):
        x, xs, xd = _rows(n, K, kind, g)
        dt = torch.float32 if kind == "f32" else torch.bfloat16
        buf = torch.full((n * O + 512,), 7.0, dtype=dt, device="cuda")  # 256 elements on either side
        y = buf[256:256 + n * O].view(n, O)
        muir.w4_matvec(x, *packed, O, x_scale=xs, y=y)
        ref, A = xd @ W.mT, xd.abs() @ W.abs().mT
        tol = (K + 16) * 2.0 ** -24 * A + (2.0 ** -8 * ref.abs() if dt == torch.bfloat16 else 0.0) + 1e-30
        assert ((y.double() - ref).abs() <= tol).all(), n
        assert (buf[:256] == 7).all() and (buf[256 + n * O:] == 7).all()
    assert muir.device_status() == 0
