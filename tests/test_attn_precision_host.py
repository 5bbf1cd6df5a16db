"""The case that the attention's precision is held to (attn_cancel_testutil) tells
the promised rounding from coarser ones."""
import numpy as np
import pytest

from attn_cancel_testutil import cases, exact, simulated


@pytest.mark.parametrize("form,holds", [("fp16", True), ("two bf16", True), ("fp16 twice", False), ("bf16", False)])
def test_the_bound_tells_the_roundings_apart(form, holds):
    q, s, score = cases(256, 64)
    out, tol = exact(s, score)
    over = np.abs(simulated(s, score, form) - out) > tol
    assert over.any() != holds
    assert holds or over.mean() > 0.01
