"""What the binding and the library refuse before a device is touched: outputs
that are too small for what a call writes, scales that overflow."""
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


@pytest.mark.parametrize("scale,ok", [(2.0 ** 127, True), (2.0 ** 127 * 1.0001, False), (2.9e38, False), (1e-38, True)])
def test_attention_scales_whose_base_2_form_overflows(scale, ok):
    """scale * log2(e) has to be a binary32 number: without one every score was NaN."""
    from nvfp4_w4a4_quantized_03_b200 import build
    from tests.test_kv_abi import _attend
    build.build()
    if ok:                                   # passes this check and stops at the next one
        assert _attend(mq.lib(), scale=scale, ws=None) == -5
    else:
        assert _attend(mq.lib(), scale=scale, ws=None) == -1
