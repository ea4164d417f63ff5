"""The fp64 oracle of the distillation where the teacher's logits lie far from 0 (no GPU)."""
import numpy as np
import pytest

from oracle import step_oracle as S


@pytest.mark.parametrize("far", [2.0**40, -(2.0**60), float(np.finfo(np.float32).min), 1e300])
def test_logits_moved_together(far):
    """Entries that are alike have the same probability wherever they lie, and one far below the
    others none."""
    ids = np.array([[3, 5, 7, -1], [1, 2, 3, 4]])
    t = np.full((2, 4), far)
    t[1, 2:] = 1.5 * far if far < 0 else far / 2
    q, logq, valid = S.teacher(ids, t, 0.5, 9)
    np.testing.assert_allclose(q, [[1 / 3] * 3 + [0], [0.5, 0.5, 0, 0]], rtol=1e-15)
    assert valid.all() and np.allclose(logq[0, :3], -np.log(3))
    r = np.random.RandomState(1)
    X, W = r.randn(2, 5), r.randn(9, 5)
    for call in (S.distill_forward, S.distill_backward):
        got, want = call(X, W, ids, t, 0.5), call(X, W, ids, np.where(t == far, 0.0, -np.inf), 0.5)
        for a, b in zip(got, want):
            np.testing.assert_allclose(a, b, rtol=1e-13, atol=1e-15)
