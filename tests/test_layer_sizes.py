"""Sizes past 32 bits are refused before they reach the C ABI, which holds them in 32
bits (on meta tensors and fake addresses: nothing is allocated, nothing reaches the GPU)."""
import ctypes as C

import pytest
import torch

import gated_delta_rule_muir_b200 as muir
from gated_delta_rule_muir_b200 import _native as N

FAKE = C.c_void_p(1 << 20)
BIG = 1 << 32


def _m(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: muir.lin_attn_fwd(_m(1, 1, 1, BIG + 64), _m(1, 1, 1, BIG + 64), _m(1, 1, 1, 64), _m(1)),
    lambda: muir.lin_attn_fwd(_m(1, 1, 1, 64), _m(1, 1, 1, 64), _m(1, 1, 1, BIG + 64), _m(1)),
    lambda: muir.lin_attn_bwd(_m(1, 1, BIG + 1, 32), _m(1, 1, BIG + 1, 32), _m(1, 1, BIG + 1, 32), _m(BIG + 1), _m(1, 1, BIG + 1, 32)),
    lambda: muir.lin_attn_workspace_bytes(_m(1, 1, 1, BIG + 64), _m(1, 1, 1, BIG + 64), _m(1, 1, 1, 64), _m(1)),
    lambda: muir.lin_attn_step(_m(1, 1, BIG + 64, 32), _m(1, 1, BIG + 64), _m(1, 1, BIG + 64), _m(1, 1, 32), _m(1)),
    lambda: muir.rms_norm(_m(1, BIG + 8), _m(BIG + 8)),
    lambda: muir.rms_norm_quant(_m(1, BIG + 8), _m(BIG + 8)),
    lambda: muir.rms_norm_bwd(_m(1, BIG + 8), _m(1, BIG + 8), _m(BIG + 8), _m(1)),
    lambda: muir.w4_quantize(_m(1, BIG + 128)),
    lambda: muir.w4_quantize(_m(BIG + 1, 128)),
    lambda: muir.w4_pack(_m(1, BIG + 128, dtype=torch.uint8), _m(1, (BIG + 128) // 128, dtype=torch.bfloat16)),
    lambda: muir.w4_matvec(_m(1, BIG + 128), _m(1, (BIG + 128) // 128, 1024, dtype=torch.uint8),
                           _m(1, (BIG + 128) // 128, 1, 16, dtype=torch.bfloat16), 16),
    lambda: muir.w4_matvec(_m(1, 128), _m(BIG // 16 + 1, 1, 1024, dtype=torch.uint8),
                           _m(BIG // 16 + 1, 1, 1, 16, dtype=torch.bfloat16), BIG + 16),
])
def test_the_binding_refuses_sizes_past_32_bits(call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()


def test_outputs_that_do_not_fill_whole_tiles_below_32_bits():
    from gated_delta_rule_muir_b200 import build
    build.build()
    lib = N.load()
    top = (1 << 31) - 1
    sb = C.c_size_t(0)
    assert lib.muir_w4_bytes(128, top - 15, 128, C.byref(sb)) == (top - 15) * 64
    for O in (top - 14, top):
        assert lib.muir_w4_bytes(128, O, 128, C.byref(sb)) == 0
        assert lib.muir_w4_quantize(FAKE, FAKE, FAKE, 128, O, 128, N.MUIR_F32, None) == N.MUIR_ERR_UNSUPPORTED
        assert lib.muir_w4_pack(FAKE, FAKE, FAKE, FAKE, 128, O, 128, None) == N.MUIR_ERR_UNSUPPORTED
        assert lib.muir_w4_matvec(FAKE, None, FAKE, FAKE, FAKE, 1, 128, O, 128, N.MUIR_BF16, N.MUIR_BF16, None) == N.MUIR_ERR_UNSUPPORTED
