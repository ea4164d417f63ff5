"""Shapes that the autograd entries refuse, with what is wrong with them (no GPU needed)."""
import pytest


@pytest.mark.parametrize("bad", [(4, 64), (2, 3, 4, 64), (64,)], ids=str)
def test_rope_says_what_shape_it_takes(bad):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    good, bad, inv = torch.zeros(4, 2, 64), torch.zeros(bad), torch.ones(32, dtype=torch.float64)
    for q, k, name in ((bad, good, "q"), (good, bad, "k")):
        with pytest.raises(ValueError, match=rf"{name} must be \[tokens, heads, head_dim\]"):
            B.rope(q, k, inv)
