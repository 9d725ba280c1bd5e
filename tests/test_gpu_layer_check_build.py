"""The layer operators in the checking build: no index outside its bounds, and the outputs
bit for bit those of the ordinary build. The child process loads the checking build
through the package's own binding (MUIR_LIBRARY) and compares with what the parent saved."""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from gated_delta_rule_muir_b200 import _native as N

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def outputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    out = []
    for dtype in (torch.float32, torch.bfloat16):
        for B, T, H, dk, dv in ((2, 300, 2, 64, 128), (1, 2100, 1, 128, 64), (3, 17, 2, 32, 32)):
            q, k, v, dy = (rand(B, T, H, d).to(dtype) for d in (dk, dk, dv, dv))
            S0, ld = rand(B, H, dk, dv), -torch.rand(H, generator=g, device="cuda")
            L = torch.tensor([T, T // 2, 0][:B], dtype=torch.int32, device="cuda")
            for state in (True, False):
                y, S = muir.lin_attn_fwd(q, k, v, ld, lengths=L, S0=S0, want_state=state)
                out += [y] + ([S] if state else [])
                out += [x for x in muir.lin_attn_bwd(q, k, v, ld, dy, lengths=L, S0=S0, want_dS0=state).values() if x is not None]
            out.append(muir.lin_attn_step(S0, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), ld))
        for n, d in ((9, 264), (33, 2048), (2, 16384)):
            x, w = rand(n, d).to(dtype), rand(d)
            f = muir.rms_norm(x, w, residual=x)
            out += [*f.values(), *muir.rms_norm_bwd(x, f["h"], w, f["rstd"], dh=x)]
            qn = muir.rms_norm_quant(x, w)
            out += [qn["q"].float(), qn["scale"]]
        codes, scales = muir.w4_quantize(rand(37, 256).to(dtype), group=64)
        out.append(muir.w4_matvec(rand(9, 256).to(dtype), *muir.w4_pack(codes, scales), 37))
    codes, scales = muir.w4_quantize(rand(37889, 128))
    out.append(muir.w4_matvec(rand(3, 128).to(torch.float8_e4m3fn), *muir.w4_pack(codes, scales), 37889))
    torch.cuda.synchronize()
    assert muir.device_status() == 0
    return [x.cpu() for x in out]


CHILD = r'''
import sys, torch
sys.path.insert(0, sys.argv[1])
from gated_delta_rule_muir_b200 import _native as N
from tests.test_gpu_layer_check_build import outputs
assert N.LIB_PATH.endswith("libmuir_check.so"), N.LIB_PATH
got, want = outputs(), torch.load(sys.argv[2])
assert len(got) == len(want)
for i, (a, b) in enumerate(zip(got, want)):
    assert torch.equal(a, b), i
print("CHECK_BUILD_OK")
'''


def test_checking_build_runs_clean(cuda_ok, tmp_path):
    assert os.path.exists(N.CHECK_LIB_PATH), "libmuir_check.so is built by __graft_entry__.build()"
    saved = str(tmp_path / "outputs.pt")
    torch.save(outputs(), saved)
    res = subprocess.run([sys.executable, "-c", CHILD, ROOT, saved], env=dict(os.environ, MUIR_LIBRARY=N.CHECK_LIB_PATH),
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0 and "CHECK_BUILD_OK" in res.stdout, res.stdout[-3000:] + res.stderr[-3000:]
