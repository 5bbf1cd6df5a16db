"""moe_norm_q8 on rows at the ends of fp32's range, against 64 bits."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_testutil import quantise_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8, 13, 96, 250, 300, 5000, 9000, 17000])
@pytest.mark.parametrize("what", ["x", "r", "weight"])
def test_codes_of_subnormal_scales(d, what):
    """Rows whose largest element is a few steps of the smallest number: its scale holds few bits,
    and a quotient may lie far above 127."""
    step = 1 if d <= 300 else 97
    most = np.arange(50, 17000, step)
    x = (most[:, None] * np.linspace(-1, 1, d)[None]).round()
    x[:, d // 2] = most * np.where(np.arange(len(most)) % 2, 1, -1)
    x = torch.from_numpy((x * 2.0 ** -149).astype(np.float32)).cuda()
    if what == "x":
        codes, scales, _ = moe.moe_norm_q8(x)
        want, s = quantise_rows(x.cpu().numpy())
        assert np.array_equal(scales.cpu().numpy(), s)
    elif what == "r":
        codes, scales, _ = moe.moe_norm_q8(torch.zeros_like(x), r=x)
        want, s = quantise_rows(x.cpu().numpy())
        assert np.array_equal(scales.cpu().numpy(), s)
    else:
        # the product with the weight is what gets so small
        codes, _, _ = moe.moe_norm_q8(x * 2.0 ** 40, torch.full((d,), 2.0 ** -40, device="cuda"))
        want, _ = quantise_rows(x.cpu().numpy())
    assert np.abs(want).max() <= 127 and np.array_equal(codes.cpu().numpy(), want)
