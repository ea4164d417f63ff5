"""The fp64 oracle of the attention and of the head norm: its gradients against
central differences of its forward, and its masks against a dense softmax."""
import numpy as np
import pytest

from oracle import attn_oracle as A

# A central difference at step h of a smooth function is off by h^2 / 6 of its
# third derivative plus rounding 1e-16 / h: at 1e-5 both are below 1e-9 here.
H, TOL = 1e-5, 1e-7


def check_gradient(f, x, grad, rng):
    for _ in range(4):
        u = rng.standard_normal(x.shape)
        want = (f(x + H * u) - f(x - H * u)) / (2 * H)
        assert abs(want - float((grad * u).sum())) <= TOL * (1 + abs(want))


@pytest.mark.parametrize("cu", [[0, 9], [0, 1, 1, 6, 9], [2, 5, 8]])
def test_attention_gradients_against_differences(cu):
    rng = np.random.default_rng(3)
    q, g = rng.standard_normal((2, 9, 4, 8))
    k, v = rng.standard_normal((2, 9, 2, 8))
    f = lambda q, k, v: float((A.attention_forward(q, k, v, cu, 0.4)[0] * g).sum())  # noqa: E731
    dq, dk, dv = A.attention_backward(g, q, k, v, cu, 0.4)
    check_gradient(lambda x: f(x, k, v), q, dq, rng)
    check_gradient(lambda x: f(q, x, v), k, dk, rng)
    check_gradient(lambda x: f(q, k, x), v, dv, rng)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [8, 16])
def test_norm_gradients_against_differences(rot, interleaved):
    rng = np.random.default_rng(5)
    x, g = rng.standard_normal((2, 7, 3, 16))
    w = 1 + 0.1 * rng.standard_normal(16)
    angle = rng.uniform(0, 6, (20, rot // 2))
    pos = rng.integers(0, 20, 7)
    a = (np.cos(angle), np.sin(angle), pos, 1e-6, interleaved)
    dx, dw = A.qk_norm_rope_backward(g, x, w, *a)
    check_gradient(lambda t: float((A.qk_norm_rope_forward(t, w, *a) * g).sum()), x, dx, rng)
    check_gradient(lambda t: float((A.qk_norm_rope_forward(x, t, *a) * g).sum()), w, dw, rng)


def test_attention_matches_dense_masked_softmax():
    rng = np.random.default_rng(7)
    q = rng.standard_normal((11, 2, 8))
    k, v = rng.standard_normal((2, 11, 1, 8))
    cu = [1, 4, 4, 10]
    of = np.array([-1, 0, 0, 0, 2, 2, 2, 2, 2, 2, -1])
    out, lse = A.attention_forward(q, k, v, cu, 0.3)
    for h in range(2):
        s = 0.3 * q[:, h] @ k[:, 0].T
        seen = (of[:, None] == of[None]) & (of[:, None] >= 0) & (np.arange(11)[:, None] >= np.arange(11))
        e = np.where(seen, np.exp(s), 0.0)
        l = e.sum(1)
        want = np.where(l[:, None] > 0, e @ v[:, 0] / np.where(l, l, 1)[:, None], 0.0)
        assert np.allclose(out[:, h], want, atol=1e-12)
        with np.errstate(divide="ignore"):
            assert np.allclose(lse[h], np.log(l), atol=1e-12)


def test_descending_offsets_leave_every_row_empty():
    rng = np.random.default_rng(9)
    q, k, v = rng.standard_normal((3, 6, 1, 8))
    out, lse = A.attention_forward(q, k, v, [0, 5, 3], 1.0)
    assert not out.any() and np.isneginf(lse).all()
