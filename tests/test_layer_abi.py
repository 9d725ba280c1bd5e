"""Refusals of the layer operators, before anything reaches the GPU: the C entry points by
their codes, the Python binding by its exceptions."""
import ctypes as C

import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from gated_delta_rule_muir_b200 import _native as N

FAKE = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_muir_b200 import build
    build.build()
    return N.load()


def _lin(**kw):
    a = N.LinArgs(B=2, T=300, H=2, dk=64, dv=32, dtype=N.MUIR_F32, flags=0, scale=1.0, q=FAKE, k=FAKE, v=FAKE,
                  log_decay=FAKE, lengths=None, S0=None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _grads(**kw):
    g = N.LinGrads(dy=FAKE, dS_T=None, dq=FAKE, dk=FAKE, dv=FAKE, dS0=None)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("field,value,code", [
    ("dk", 48, N.MUIR_ERR_UNSUPPORTED), ("dv", 256, N.MUIR_ERR_UNSUPPORTED), ("H", 0, N.MUIR_ERR_UNSUPPORTED),
    ("dtype", N.MUIR_E4M3, N.MUIR_ERR_UNSUPPORTED), ("B", 40000, N.MUIR_ERR_UNSUPPORTED),
    ("T", 1 << 31, N.MUIR_ERR_UNSUPPORTED), ("B", -1, N.MUIR_ERR_INVALID_ARG), ("T", -1, N.MUIR_ERR_INVALID_ARG),
    ("flags", 1, N.MUIR_ERR_INVALID_ARG), ("q", None, N.MUIR_ERR_INVALID_ARG), ("v", ODD, N.MUIR_ERR_INVALID_ARG),
    ("log_decay", None, N.MUIR_ERR_INVALID_ARG), ("S0", ODD, N.MUIR_ERR_INVALID_ARG),
    ("lengths", C.c_void_p((1 << 20) + 2), N.MUIR_ERR_INVALID_ARG),
])
def test_lin_refusals(lib, field, value, code):
    a = _lin(**{field: value})
    assert lib.muir_lin_fwd(C.byref(a), FAKE, None, FAKE, 1 << 40, None) == code
    assert lib.muir_last_error()
    g = _grads()
    assert lib.muir_lin_bwd(C.byref(a), C.byref(g), FAKE, 1 << 40, None) == code


def test_lin_outputs_and_workspaces(lib):
    for dtype in (N.MUIR_F32, N.MUIR_BF16):
        a = _lin(B=1, T=100000, dtype=dtype)
        assert lib.muir_lin_fwd(C.byref(a), None, None, FAKE, 1 << 40, None) == N.MUIR_ERR_INVALID_ARG
        assert lib.muir_lin_fwd(C.byref(a), FAKE, ODD, FAKE, 1 << 40, None) == N.MUIR_ERR_INVALID_ARG
        need = lib.muir_lin_fwd_workspace(C.byref(a))
        assert need > 0
        assert lib.muir_lin_fwd(C.byref(a), FAKE, None, FAKE, need - 1, None) == N.MUIR_ERR_WORKSPACE
        assert lib.muir_lin_fwd(C.byref(a), FAKE, None, None, need, None) == N.MUIR_ERR_WORKSPACE
        assert lib.muir_lin_fwd(C.byref(a), FAKE, None, C.c_void_p((1 << 20) + 16), need, None) == N.MUIR_ERR_WORKSPACE
        need = lib.muir_lin_bwd_workspace(C.byref(a))
        for f in ("dy", "dq", "dk", "dv"):
            g = _grads(**{f: None})
            assert lib.muir_lin_bwd(C.byref(a), C.byref(g), FAKE, need, None) == N.MUIR_ERR_INVALID_ARG
        g = _grads()
        assert lib.muir_lin_bwd(C.byref(a), C.byref(g), FAKE, need - 1, None) == N.MUIR_ERR_WORKSPACE
        assert lib.muir_lin_bwd(C.byref(a), None, FAKE, need, None) == N.MUIR_ERR_INVALID_ARG
    a = _lin(B=0, q=None, k=None, v=None, log_decay=None)
    assert lib.muir_lin_fwd(C.byref(a), None, None, None, 0, None) == N.MUIR_OK
    assert lib.muir_lin_bwd(C.byref(a), C.byref(_grads()), None, 0, None) == N.MUIR_OK
    assert lib.muir_lin_fwd(None, FAKE, None, None, 0, None) == N.MUIR_ERR_INVALID_ARG


def test_lin_step_refusals(lib):
    def call(**kw):
        a = N.LinStepArgs(n_seq=2, H=2, dk=64, dv=32, dtype=N.MUIR_BF16, scale=1.0, S=FAKE, q=FAKE, k=FAKE, v=FAKE,
                          log_decay=FAKE, y=FAKE)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.muir_lin_step(C.byref(a), None)
    assert call(n_seq=0, S=None) == N.MUIR_OK
    assert call(n_seq=-1) == N.MUIR_ERR_INVALID_ARG
    assert call(dk=33) == N.MUIR_ERR_UNSUPPORTED
    assert call(dtype=2) == N.MUIR_ERR_UNSUPPORTED
    assert call(n_seq=1 << 40) == N.MUIR_ERR_UNSUPPORTED
    for f in ("S", "q", "k", "v", "log_decay", "y"):
        assert call(**{f: None}) == N.MUIR_ERR_INVALID_ARG
        assert call(**{f: ODD}) == N.MUIR_ERR_INVALID_ARG
    assert lib.muir_lin_step(None, None) == N.MUIR_ERR_INVALID_ARG


def test_norm_refusals(lib):
    def call(x=FAKE, res=None, w=FAKE, y=FAKE, h=None, n=4, d=64, eps=1e-6, dt=N.MUIR_BF16):
        return lib.muir_rms_norm(x, res, w, y, h, None, n, d, eps, dt, None)

    def quant(x=FAKE, q=FAKE, scale=FAKE, res=None, h=None, d=64):
        return lib.muir_rms_norm_quant(x, res, FAKE, q, scale, h, None, 4, d, 1e-6, N.MUIR_F32, None)
    assert call(n=0, x=None) == N.MUIR_OK
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(res=FAKE), dict(x=ODD), dict(n=-1), dict(eps=-1.0),
               dict(eps=float("nan"))):
        assert call(**kw) == N.MUIR_ERR_INVALID_ARG, kw
    for kw in (dict(d=0), dict(d=60), dict(d=16392), dict(dt=2), dict(n=1 << 33)):
        assert call(**kw) == N.MUIR_ERR_UNSUPPORTED, kw
    for kw in (dict(q=None), dict(scale=None), dict(res=FAKE), dict(scale=C.c_void_p((1 << 20) + 1))):
        assert quant(**kw) == N.MUIR_ERR_INVALID_ARG, kw

    def bwd(dy=FAKE, h=FAKE, w=FAKE, r=FAKE, dx=FAKE, dw=FAKE, n=4, d=64, ws=FAKE, nb=1 << 30):
        return lib.muir_rms_norm_bwd(dy, h, w, r, None, dx, dw, n, d, N.MUIR_F32, ws, nb, None)
    for f in ("dy", "h", "w", "r", "dx", "dw"):
        assert bwd(**{f: None}) == N.MUIR_ERR_INVALID_ARG, f
    need = lib.muir_rms_norm_bwd_workspace(4, 64)
    assert need > 0
    assert bwd(nb=need - 1) == N.MUIR_ERR_WORKSPACE and bwd(ws=None) == N.MUIR_ERR_WORKSPACE
    assert bwd(d=4) == N.MUIR_ERR_UNSUPPORTED and lib.muir_rms_norm_bwd_workspace(4, 4) == 0


def test_w4_refusals(lib):
    def call(x=FAKE, xs=None, wq=FAKE, ws=FAKE, y=FAKE, n=4, K=256, O=33, g=64, xd=N.MUIR_BF16, yd=N.MUIR_BF16):
        return lib.muir_w4_matvec(x, xs, wq, ws, y, n, K, O, g, xd, yd, None)
    assert call(n=0, x=None) == N.MUIR_OK
    for kw in (dict(x=None), dict(wq=None), dict(ws=ODD), dict(y=None), dict(n=-1), dict(xs=FAKE)):
        assert call(**kw) == N.MUIR_ERR_INVALID_ARG, kw
    for kw in (dict(K=192), dict(K=0), dict(O=0), dict(g=16), dict(xd=N.MUIR_F32), dict(yd=2), dict(xd=3), dict(n=1 << 40)):
        assert call(**kw) == N.MUIR_ERR_UNSUPPORTED, kw
    sb = C.c_size_t(7)
    assert lib.muir_w4_bytes(256, 33, 64, C.byref(sb)) == 48 * 128 and sb.value == 48 * 4 * 2
    assert lib.muir_w4_bytes(100, 33, 64, C.byref(sb)) == 0 and sb.value == 0
    assert lib.muir_w4_pack(FAKE, FAKE, None, FAKE, 256, 33, 64, None) == N.MUIR_ERR_INVALID_ARG
    assert lib.muir_w4_pack(FAKE, FAKE, FAKE, FAKE, 256, 33, 48, None) == N.MUIR_ERR_UNSUPPORTED
    assert lib.muir_w4_quantize(FAKE, None, FAKE, 256, 33, 64, N.MUIR_F32, None) == N.MUIR_ERR_INVALID_ARG
    assert lib.muir_w4_quantize(FAKE, FAKE, FAKE, 256, 33, 64, 2, None) == N.MUIR_ERR_UNSUPPORTED


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros
    q, v, ld = z(1, 4, 2, 32), z(1, 4, 2, 32), z(2)
    with pytest.raises(ValueError, match="CUDA"):
        muir.lin_attn_fwd(q, q, v, ld)
    with pytest.raises(ValueError, match="dimensions"):
        muir.lin_attn_fwd(q[0], q, v, ld)
    with pytest.raises(TypeError, match="float16"):
        muir.lin_attn_fwd(q.half(), q.half(), v.half(), ld)
    with pytest.raises(ValueError, match="CUDA"):
        muir.lin_attn_step(z(1, 2, 32, 32), z(1, 2, 32), z(1, 2, 32), z(1, 2, 32), ld)
    with pytest.raises(ValueError, match="CUDA"):
        muir.rms_norm(z(2, 8), z(8))
    with pytest.raises(ValueError, match="CUDA"):
        muir.rms_norm_bwd(z(2, 8), z(2, 8), z(8), z(2))
    with pytest.raises(ValueError, match="multiple of 128"):
        muir.w4_pack(z(4, 100, dtype=torch.uint8), z(4, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="tiles"):
        muir.w4_matvec(z(1, 128), z(1, 1, 1024, dtype=torch.uint8), z(1, 1, 1, 16, dtype=torch.bfloat16), 17)


def test_the_binding_takes_its_operands_by_name_and_only_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="x: must be a contiguous CUDA tensor"):
        muir.rms_norm(weight=z(8), x=z(2, 8))
    for bad in (None, [1.0], 3):
        with pytest.raises(TypeError, match="expected a tensor"):
            muir.rms_norm(bad, z(8))
    with pytest.raises(TypeError, match="expected a tensor"):
        muir.w4_matvec()
