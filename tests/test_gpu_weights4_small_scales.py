"""Quantising the smallest groups.  A scale that is a bf16 subnormal is a whole number of
steps of 2^-133, up to half a step from max |w| / 7: with the largest at 8 steps it is
one step, and the quotients reach 8.  The codes are those of the 64-bit form, whose
quotients are limited to -8..7 (equal)."""
import pytest
import torch

from tests import weights4_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _quantize(W, segments, group):
    """codes [rows, cols] and scales, in 64 bits."""
    q, scales = ref.quantize(W, segments, group)
    return q.clamp(0, 15), scales


# pieces of 16 elements; eight columns to a thread; a byte to a thread, segments of less than eight
@pytest.mark.parametrize("cols,segments", [(128, 1), (256, 2), (99, 1), (100, 5), (21, 3), (10, 2)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_codes_of_the_smallest_groups(cols, segments, group):
    from megatron_tensor_transformer_w1_gb300 import weights4 as w4
    g = torch.Generator(device="cuda").manual_seed(cols + group)
    top = torch.arange(1, 301, device="cuda").repeat(4)[:, None]
    steps = (torch.rand(1200, cols, generator=g, device="cuda") * (2 * top + 1)).floor() - top
    largest = torch.where(torch.arange(1200, device="cuda") % 600 < 300, 1, -1)[:, None] * top
    steps[:, ::7] = largest.float()  # in every group, at even and odd columns
    W = (steps.double() * 2.0 ** -133).to(BF)
    # ordinary groups beside them: a row's largest are of both kinds
    W[600:, cols // 2:] = torch.randn(600, cols - cols // 2, generator=g, device="cuda").to(BF)
    c = w4.quantize4(W, group=group, segments=segments)
    q, scales = _quantize(W, segments, group)
    assert torch.equal(c.scales, scales)
    assert torch.equal(ref.nibbles(c.codes, cols), q)
    assert torch.equal(w4.dequantize4(c), ref.matrix(c.codes, c.scales, cols, segments, group).to(BF))
