"""What the binding refuses by itself, before the library or a device is
touched: outputs that are too small for what a call writes."""
import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import mq

X = torch.zeros(4, 64, dtype=torch.bfloat16)
U8 = torch.zeros(1 << 16, dtype=torch.uint8)
ALPHA = torch.ones(1)


@pytest.mark.parametrize("y", [torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(4 * 128 - 1, dtype=torch.bfloat16),
                               torch.zeros(4, 128)])
def test_linear_outputs_too_small(y):
    with pytest.raises(AssertionError):
        mq.mq_linear_w4a4(X, U8, U8, ALPHA, 128, y, U8)


@pytest.mark.parametrize("y", [torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(4, 128)])
def test_mlp_outputs_too_small(y):
    with pytest.raises(AssertionError):
        mq.mq_mlp_w4a4(X, U8, U8, ALPHA, 64, U8, U8, ALPHA, 128, y, U8)
