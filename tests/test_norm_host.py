"""Refusals of the head norm that depend on more than one argument: no GPU needed."""
import ctypes

import pytest

from tests.test_attention_host import B, P, norm_desc  # noqa: F401


@pytest.mark.parametrize("rot_dim", [0, 64])
def test_positions_are_aligned(B, rot_dim):  # noqa: F811
    """They are read without a rotation too."""
    d = ctypes.byref(norm_desc(B, rot_dim=rot_dim))
    args = [P] * 10
    args[6] = P + 4
    assert B.lib().flce_qk_norm_rope_forward(d, *args, None) == B.FLCE_ERR_ARG
    args = [P] * 11
    args[8] = P + 4
    assert B.lib().flce_qk_norm_rope_backward(d, *args, P, P, P, 1 << 30, P, None) == B.FLCE_ERR_ARG
