"""Sizes past 32 bits are refused before they reach the C ABI, which holds them in 32
bits (on meta tensors: nothing is allocated, nothing reaches the GPU)."""
import pytest
import torch

import gated_delta_rule_muir_b200 as muir

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
