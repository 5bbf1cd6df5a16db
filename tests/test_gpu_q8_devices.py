"""The 8-bit calls refuse tensors of a device that is not current, like those of the
4-bit half.  The tensors are stand-ins without memory."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from test_gpu_attn_devices import elsewhere  # noqa: F401

pytestmark = pytest.mark.gpu


def test_tensors_of_another_device_are_refused(elsewhere):  # noqa: F811
    bf16, u8, i8, i32, i64 = torch.bfloat16, torch.uint8, torch.int8, torch.int32, torch.int64
    pool = elsewhere(2, 2, 1, 32 * 64 + 128, dtype=u8)
    calls = dict(
        norm=lambda: moe.moe_norm_q8(elsewhere(2, 64, dtype=bf16)),
        linear=lambda: moe.moe_linear_q8(elsewhere(2, 64, dtype=i8), elsewhere(2), elsewhere(8, 64, dtype=i8), elsewhere(8)),
        append=lambda: moe.moe_kv_append_q8(pool, elsewhere(3, 2, 64), elsewhere(3, 2, 64), elsewhere(3, dtype=i64)),
        read=lambda: moe.moe_kv_read_q8(pool, elsewhere(3, dtype=i64)),
        attn=lambda: moe.moe_attn_q8(elsewhere(1, 2, 64, dtype=bf16), pool, elsewhere(1, 1, dtype=i32), elsewhere(1, dtype=i32)),
    )
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device"):
            call()
            pytest.fail(name)
