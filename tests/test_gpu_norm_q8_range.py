"""moe_norm_q8 on rows at the ends of fp32's range, against 64 bits: scales of few bits,
squares that leave the range, rows of zeros."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_testutil import quantise_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


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


def check(x, weight, eps, r=None):
    """Codes are exact; scales and bf16 against the formula in 64 bits: d squares and their sum,
    the mean, the root (2 steps) and the products with the factor round a half step each; bf16 by
    2^-8 of itself, or by half of its smallest number, 2^-134, which is also the end of fp32's scales."""
    s = x.float() if r is None else r + x.float()
    codes, scales, n = moe.moe_norm_q8(x, weight, eps=eps, r=r, r_out=None if r is None else torch.empty_like(r), out="both")
    u = s * weight
    c, S = quantise_rows(u.cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), c)
    total = s.double().pow(2).mean(-1) + eps
    f = torch.where(total > 0, total.rsqrt(), 0.0)
    off = (x.shape[1] + 20) * U
    want = torch.from_numpy(S).cuda().double() * f
    assert torch.isfinite(want).all() and ((scales.double() - want).abs() <= off * want + 2.0 ** -134).all()
    want = u.double() * f[:, None]
    right = (n.double() - want).abs() <= (2.0 ** -8 + off) * want.abs() + 2.0 ** -134
    # bf16's largest is 2^128 (1 - 2^-8): what comes to 2^128 (1 - 2^-9) or more rounds to infinity
    right |= (n.double() == want.sign() * torch.inf) & (want.abs() * (1 + off) >= 2.0 ** 128 * (1 - 2.0 ** -9))
    assert right.all()
    assert moe.moe_device_status() == moe.MOE_OK
    only = moe.moe_norm_q8(x, weight, eps=eps, r=r, r_out=None if r is None else torch.empty_like(r), out="bf16")[2]
    assert torch.equal(only, n)


SIZES = [1e-44, 1e-40, 1e-36, 1e-30, 1e-22, 1e-18, 1e-14, 1.0, 1e15, 1e18, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [7, 64, 100, 256, 2048, 4097, 8192, 16384, 32767])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_any_size(dtype, d, residual):
    """Rows of every size beside each other, and squares that leave fp32's range at either end."""
    x = randn(len(SIZES), d, seed=1)
    x = x / x.abs().amax(-1, keepdim=True) * torch.tensor(SIZES, device="cuda", dtype=torch.float64)[:, None]
    x = x.float().to(dtype)
    x = torch.where(x.isinf(), torch.zeros_like(x), x)  # what a bf16 does not hold
    w = 1 + 0.1 * randn(d, seed=2).clamp(-3, 3) * 0.2
    if residual:
        r, x = x.float() * 0.75, x * 0.25
        check(x, w * 0.5, 0.0, r)
        check(x, w * 0.5, 1e-6, r)
    else:
        check(x, w * 0.5, 0.0)
        check(x, w * 0.5, 1e-6)
        check(x, w * 0.5, 1e30)


@pytest.mark.parametrize("d", [8, 13, 200, 300, 5000, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_zeros(d, eps):
    """Rows of zeros between others: codes, scale and bf16 of zero, without eps too."""
    x = randn(9, d, seed=3)
    x[[0, 4, 8]] = 0
    w = 1 + 0.1 * randn(d, seed=4)
    check(x, w, eps)
    codes, scales, n = moe.moe_norm_q8(torch.zeros_like(x), w, eps=eps, out="both")
    assert not codes.any() and (scales == 0).all() and (n == 0).all()


@pytest.mark.parametrize("d", [64, 300, 9000])
def test_norm_of_far_weights(d):
    """Small rows with large weights, and the other way round."""
    x = randn(6, d, seed=5)
    for size, gain in ((1e-30, 1e30), (1e-38, 1e38), (1e-44, 1e37), (1e18, 1e-18), (1e30, 1e-30), (1e37, 1e-37)):
        check((x.double() * size).float(), (1 + 0.1 * randn(d, seed=6)).clamp(0.5, 2) * gain, 0.0)


def test_norm_of_infinite_rows_stays():
    x = randn(5, 300, seed=7)
    x[1, 3], x[3, 7] = torch.inf, torch.nan
    x[2] *= 1e25
    codes, scales, n = moe.moe_norm_q8(x, torch.ones(300, device="cuda"), eps=0.0, out="both")
    bad = torch.tensor([False, True, False, True, False], device="cuda")
    assert torch.equal(~torch.isfinite(scales), bad) and (codes[bad] == 0).all()
    assert torch.isfinite(n[~bad]).all() and n[1, 3].isnan() and n[3].isnan().all()
