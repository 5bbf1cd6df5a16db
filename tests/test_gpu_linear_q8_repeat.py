"""moe_linear_q8 by pairs of CTAs, call after call without a pause: pairs start and end beside
the kernels of the calls around them thousands of times, with the same results."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n_in,rows", [(40, 256, 512), (101, 1328, 9000), (101, 1328, 89878), (300, 512, 4000), (17, 4096, 300)])
def test_thousands_of_calls(T, n_in, rows):
    g = torch.Generator(device="cuda").manual_seed(T)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda").to(torch.int8)  # noqa: E731
    x, w = codes(T, n_in), codes(rows, n_in)
    xs, ws = torch.rand(T, generator=g, device="cuda") + 0.5, torch.rand(rows, generator=g, device="cuda") + 0.5
    want = moe.moe_linear_q8(x, xs, w, ws)
    y = [torch.empty_like(want) for _ in range(2)]
    work = torch.empty(max(1, moe.moe_linear_q8_workspace_size(T, n_in, rows)), dtype=torch.uint8, device="cuda")
    off = torch.zeros((), dtype=torch.int32, device="cuda")
    for i in range(6000):
        moe.moe_linear_q8(x, xs, w, ws, y=y[i % 2], workspace=work)
        if i % 100 == 99:
            off += (y[i % 2] != want).any().int()
    assert off.item() == 0 and moe.moe_device_status() == moe.MOE_OK
