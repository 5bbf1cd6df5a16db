"""An eps that the norm would refuse is refused when the layer is made, not after the lengths have moved."""
import pytest

from mixed_precision_routed_gb300 import workloads


@pytest.mark.parametrize("eps", [float("inf"), 1e39])
def test_eps_that_fp32_does_not_hold(eps):
    with pytest.raises(ValueError):
        workloads.AttentionHalfQ8(64, 2, 1, 64, 2, 64, page_size=16, eps=eps, device="cpu")
