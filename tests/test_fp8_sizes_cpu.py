"""Sizes past what the argument blocks of the 8-bit calls hold are refused: ctypes
keeps the low 32 bits of a number without a word, so K = 2^32 + 16 would reach the
library as K = 16.  Meta tensors have a shape and no memory."""
import pytest
import torch

import gated_delta_rule_150_b200 as gdr

bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LIMIT = 2 ** 31 - 1024


def _meta(*shape, dtype=f32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def _linear(rows, n, k):
    return (_meta(rows, k, dtype=e4m3), _meta(rows, -(-k // 128)), _meta(n, k, dtype=e4m3),
            _meta(-(-n // 128), -(-k // 128)))


@pytest.mark.parametrize("over", [LIMIT + 1024, 2 ** 31 + 16, 2 ** 32 + 16])
def test_sizes_past_the_limit_are_refused(over):
    with pytest.raises(ValueError, match="rows must be at most"):
        gdr.norm_fp8(_meta(over, 16, dtype=bf16), _meta(16))
    with pytest.raises(ValueError, match="rows must be at most"):
        gdr.gated_norm_fp8(_meta(over, 1, 64), _meta(over, 1, 64), _meta(64))
    with pytest.raises(ValueError, match="H . d_v must be at most"):
        gdr.gated_norm_fp8(_meta(1, over // 16, 64), _meta(1, over // 16, 64), _meta(64))
    with pytest.raises(ValueError, match="N must be at most"):
        gdr.quantize_weight_fp8(_meta(over, 16, dtype=bf16))
    with pytest.raises(ValueError, match="K must be at most"):
        gdr.quantize_weight_fp8(_meta(1, over, dtype=bf16))
    for name, sizes in (("rows", (over, 1, 16)), ("N", (1, over, 16)), ("K", (1, 1, over))):
        with pytest.raises(ValueError, match=f"{name} must be at most"):
            gdr.linear_fp8(*_linear(*sizes))


def test_sizes_at_the_limit_reach_the_device_check():
    top = LIMIT // 16 * 16
    for call in (lambda: gdr.norm_fp8(_meta(LIMIT, 16, dtype=bf16), _meta(16)),
                 lambda: gdr.quantize_weight_fp8(_meta(LIMIT, 16, dtype=bf16)),
                 lambda: gdr.quantize_weight_fp8(_meta(1, top, dtype=bf16)),
                 lambda: gdr.linear_fp8(*_linear(LIMIT, 1, 16)),
                 lambda: gdr.linear_fp8(*_linear(1, LIMIT, 16)),
                 lambda: gdr.linear_fp8(*_linear(1, 1, top))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
