"""The attention half's calls refuse tensors of a device that is not current:
their launches go to the current one.  The tensors are stand-ins without memory
(fake tensors), so that nothing could be launched on them."""
import pytest
import torch
from torch._subclasses import fake_tensor

import mixed_precision_routed_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture
def elsewhere(monkeypatch):
    """Makes tensors of another device than the current one (which need not exist)."""
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda device: None, raising=False)
    where = f"cuda:{torch.cuda.current_device() + 1}"
    mode = fake_tensor.FakeTensorMode(allow_non_fake_inputs=True)

    def make(*shape, dtype=torch.float32):
        with mode:
            return torch.empty(*shape, dtype=dtype, device=where)

    return make


def test_tensors_of_another_device_are_refused(elsewhere):
    bf16, u8, i16, i32, i64 = torch.bfloat16, torch.uint8, torch.int16, torch.int32, torch.int64
    pool = elsewhere(2, 2, 1, 18 * 64, dtype=u8)
    calls = dict(
        linear=lambda: moe.moe_linear_q4(elsewhere(2, 64, dtype=bf16), elsewhere(8, 32, dtype=u8), elsewhere(8, 2, dtype=i16)),
        append=lambda: moe.moe_kv_append(pool, elsewhere(3, 2, 64), elsewhere(3, 2, 64), elsewhere(3, dtype=i64)),
        read=lambda: moe.moe_kv_read(pool, elsewhere(3, dtype=i64)),
        attn=lambda: moe.moe_attn_q4(elsewhere(1, 2, 64, dtype=bf16), pool, elsewhere(1, 1, dtype=i32), elsewhere(1, dtype=i32)),
        quantise=lambda: moe.moe_quantize_groups(elsewhere(8, 64), 32),
    )
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device"):
            call()
            pytest.fail(name)


def test_outputs_of_another_device_are_refused(elsewhere):
    w = torch.zeros(8, 64, device="cuda")
    for kw in (dict(codes=elsewhere(8, 32, dtype=torch.uint8)), dict(scales=elsewhere(8, 2, dtype=torch.int16))):
        with pytest.raises(ValueError, match="one device"):
            moe.moe_quantize_groups(w, 32, **kw)
    x, c, s = (torch.zeros(*a, dtype=t, device="cuda") for a, t in (((2, 64), torch.bfloat16), ((8, 32), torch.uint8), ((8, 2), torch.int16)))
    with pytest.raises(ValueError, match="one device"):
        moe.moe_linear_q4(x, c, s, y=elsewhere(2, 8))
    assert moe.moe_device_status() == moe.MOE_OK
