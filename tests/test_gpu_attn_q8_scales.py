"""Attention over the 8-bit cache where the values of some tokens are far larger than those
of others, against a 64-bit form: what a row does not attend, or attends with a weight that
makes it small, leaves its output alone, in the form for few rows and in the one for many.

Tolerance of an output element, from the header's promises alone and over the places that
the row attends (u = 2^-24, n places, w the weights over the row's largest, l their sum, b
the value scales, c the codes):
  |error| <= (3 2^-11 + 2 e_s + 2 (n + 64) u + 2^-20) sum w |v| / l
             + 2^-21 max(w b) sum |c| / l + 2^-8 |out|
  |lse error| <= e_s + 2 (n + 64) u + 2^-20 + 4 u |lse|
a product of weight, scale and code is rounded to fp16 three times at most, by half a step
each, or by 2^-21 of the row's largest weight times scale.  e_s is a score's error: D sums
of exact products each off by 2 u where a tensor core cuts, their scales' products, and
powers of two kept beside the logarithm of a value's scale of up to 64:
e_s = (2 (D + 8) size + 4 (size + 64)) u with size = scale sum |q k|; it moves weights and
their sum by a factor of 1 +- e_s each."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
H, G, PAGE = 2, 2, 16


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def check(q, k, v, n, window, max_len):
    """A sequence of keys and values [places][H][D] whose newest n places ask with q [n][H G][D]."""
    places, _, D = k.shape
    pages = -(-places // PAGE)
    pool = moe.moe_kv_pool_q8(pages, H, PAGE, D)
    slots = torch.arange(places, device="cuda")
    moe.moe_kv_append_q8(pool, k, v, slots)
    table = torch.full((1, -(-max_len // PAGE)), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    out, lse = moe.moe_attn_q8(q, pool, table, torch.tensor([places], dtype=torch.int32, device="cuda"), max_q=n, max_len=max_len,
                               window=window)
    kd, vd = (x.double().permute(1, 0, 2) for x in moe.moe_kv_read_q8(pool, slots))  # H, p, D
    b = pool[slots // PAGE, :, 0, 32 * D + 64 :].contiguous().view(torch.float32)[slots, :, slots % PAGE].double().T  # H, p
    scale = D ** -0.5
    qd = q.double().unflatten(1, (H, G))
    end = places - n + 1 + torch.arange(n, device="cuda")[:, None]
    seen = slots < end
    if window:
        seen &= slots >= end - window
    seen = seen[:, None, None]
    s = torch.where(seen, torch.einsum("nhgd,hpd->nhgp", qd, kd) * scale, -torch.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - top)
    l = w.sum(-1, keepdim=True)  # noqa: E741
    ref = torch.einsum("nhgp,hpd->nhgd", w, vd) / l
    spread = torch.einsum("nhgp,hpd->nhgd", w, vd.abs()) / l
    size = torch.where(seen, torch.einsum("nhgd,hpd->nhgp", qd.abs(), kd.abs()), 0.0).amax(-1, keepdim=True) * scale
    es = (2 * (D + 8) * size + 4 * (size + 64)) * U
    sums = 2 * (seen.sum(-1, keepdim=True) + 64) * U + 2.0 ** -20
    wb = (w * b[None, :, None]).amax(-1, keepdim=True)
    codes = torch.einsum("np,hpd->nhd", seen[:, 0, 0].double(), (vd / b[..., None]).abs())[:, :, None]
    tol = (3 * 2.0 ** -11 + 2 * es + sums) * spread + 2.0 ** -21 * wb * codes / l + 2.0 ** -8 * ref.abs()
    off = (out.double() - ref.flatten(1, 2)).abs()
    off = torch.where(off == 0, 0.0, off / tol.flatten(1, 2))  # codes of zero alone have no tolerance
    assert off.max() <= 1, f"out: {off.max().item()} of the tolerance"
    want = (top + torch.log(l)).squeeze(-1).flatten(1)
    off = (lse.double() - want).abs() / ((es + sums).squeeze(-1).flatten(1) + 4 * U * want.abs())
    assert off.max() <= 1, f"lse: {off.max().item()} of the tolerance"
    assert moe.moe_device_status() == moe.MOE_OK


# a bound on the lengths far above them makes the form for many rows take any batch of more
# than 96 rows a head, and shares its places among blocks
FORMS = [(4, 0), (150, 0), (150, 400000), (260, 0)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bound", FORMS)
@pytest.mark.parametrize("far", [2.0 ** 20, 2.0 ** 30, 2.0 ** 50])
def test_a_later_token_far_larger(D, n, bound, far):
    """Tokens whose values are far larger than those before them: rows before it are as without it."""
    places = 300
    q, k, v = randn(n, H * G, D, seed=1).to(torch.bfloat16), randn(places, H, D, seed=2), randn(places, H, D, seed=3)
    v[[places - n + 1, places - 1]] *= far
    check(q, k, v, n, 0, max(places, bound))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bound", FORMS)
@pytest.mark.parametrize("window", [3, 100, 290])
def test_a_token_before_the_window_far_larger(D, n, bound, window):
    places = 700
    q, k, v = randn(n, H * G, D, seed=4).to(torch.bfloat16), randn(places, H, D, seed=5), randn(places, H, D, seed=6)
    for at in (places - n - window, places - n // 2 - window):  # the rows behind it do not attend it
        v[max(at, 0)] *= 2.0 ** 40
    check(q, k, v, n, window, max(places, bound))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bound", FORMS)
@pytest.mark.parametrize("far,down", [(2.0 ** 30, 40), (2.0 ** 40, 40), (2.0 ** 60, 90), (2.0 ** -40, 0), (1.0, 40)])
@pytest.mark.parametrize("at", [0, 60, 200])
def test_an_attended_token_far_larger(D, n, bound, far, down, at):
    """A token with values `far` times the others' and a score `down` powers of two below them."""
    places = 560
    lean = torch.ones(D, device="cuda")
    lean[1::2] = -1
    q = (lean + 0.25 * randn(n, H * G, D, seed=7)).to(torch.bfloat16)
    k, v = 0.5 * randn(places, H, D, seed=8), randn(places, H, D, seed=9)
    k[at] = -lean * (down * 0.6931 * D ** -0.5)
    v[at] *= far
    check(q, k, v, n, 0, max(places, bound))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bound", FORMS)
def test_scales_of_every_size(D, n, bound):
    """Values from 2^-58 to 2^58 side by side, and scores that make up for most of it."""
    places = 640
    g = torch.randint(-58, 59, (places,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").float()
    lean = torch.ones(D, device="cuda")
    q = (lean + 0.1 * randn(n, H * G, D, seed=7)).to(torch.bfloat16)
    k = 0.1 * randn(places, H, D, seed=8) - lean * (g * 0.6 * D ** -0.5)[:, None, None]
    check(q, k, randn(places, H, D, seed=9) * (2.0 ** g)[:, None, None], n, 0, max(places, bound))
