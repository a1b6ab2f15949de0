"""Calls of the 4-bit weights' Python layer that are refused before any device work."""
import pytest
import torch


def test_codes_in_host_memory_are_refused():
    from megatron_tensor_transformer_w1_gb300 import build
    build.build()
    from megatron_tensor_transformer_w1_gb300.weights4 import Codes4, dequantize4, quantize4
    c = Codes4(torch.zeros(3, 50, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.bfloat16), 99, group=32)
    for bad in (c, c.codes, None):
        with pytest.raises(ValueError):
            dequantize4(bad)
    with pytest.raises(ValueError):
        quantize4(torch.zeros(3, 99, dtype=torch.bfloat16))
