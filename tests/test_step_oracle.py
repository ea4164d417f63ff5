"""The fp64 oracle of layer norm, rotary positions and distillation against torch's fp64
autograd, differences and closed forms (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S

R = np.random.RandomState


@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_is_torchs(rms):
    r = R(1)
    x, w, b, g, ds = r.randn(5, 16) + 0.3, r.randn(16), r.randn(16), r.randn(5, 16), r.randn(5, 16)
    tx, tw, tb = (torch.tensor(t, requires_grad=True) for t in (x, w, b))
    y = (torch.nn.functional.rms_norm(tx, (16,), tw, 1e-3) + tb if rms
         else torch.nn.functional.layer_norm(tx, (16,), tw, tb, 1e-3))
    ((y * torch.tensor(g)).sum() + (tx * torch.tensor(ds)).sum()).backward()
    np.testing.assert_allclose(S.layer_norm_forward(x, w, b, 1e-3, rms)[0], y.detach().numpy(), atol=1e-12)
    for got, want in zip(S.layer_norm_backward(g, x, w, 1e-3, ds, rms), (tx, tw, tb)):
        np.testing.assert_allclose(got, want.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_and_turns_back(interleaved):
    r = R(2)
    x, inv, pos = r.randn(4, 3, 16), np.array([1.0, 0.3, 0.01, 1e-4]), [0, 5, -7, 10**6]
    y = S.rope(x, inv, pos, 1.0, interleaved)
    assert (y[0] == x[0]).all() and (y[..., 8:] == x[..., 8:]).all()
    np.testing.assert_allclose(S.rope(y, inv, pos, 1.0, interleaved, backward=True), x, atol=1e-12)
    # the product of two turned heads depends on the distance of their positions alone
    a, b = r.randn(2, 1, 16), r.randn(2, 1, 16)
    a[1], b[1] = a[0], b[0]
    p = (S.rope(a, inv, [3, 103], 2.0, interleaved) * S.rope(b, inv, [10, 110], 2.0, interleaved))[..., :8].sum(-1)
    assert abs(p[0] - p[1]) < 1e-12


def make(N=6, H=5, V=11, K=4, seed=3):
    r = R(seed)
    X, W, t = r.randn(N, H), r.randn(V, H), 2 * r.randn(N, K)
    ids = np.stack([r.permutation(V)[:K] for _ in range(N)])
    ids[0, 2:] = -1
    ids[1] = -1
    ids[2, 3] = ids[2, 0]  # the same id twice
    t[3, 1] = -np.inf
    return X, W, ids, t


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distillation_is_torchs(temperature, tail):
    X, W, ids, t = make()
    tl = R(4).rand(len(X)) + 3.0 if tail else None
    tX, tW = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    logp = torch.log_softmax(tX @ tW.T / temperature, -1)
    total, count = 0.0, 0
    for i in range(len(X)):
        ks = [k for k in range(ids.shape[1]) if ids[i, k] >= 0 and t[i, k] > -np.inf]
        if not ks:
            continue
        count += 1
        lq = torch.tensor(t[i, ks] / temperature)
        lq = lq - (torch.logsumexp(lq, 0) if tl is None else tl[i])
        total = total + (lq.exp() * (lq - logp[i, ids[i, ks]])).sum()
    (total / count * 0.7).backward()
    loss, rows, lse, logits, n = S.distill_forward(X, W, ids, t, temperature, teacher_lse=tl)
    assert n == count == 5 and abs(loss - total.item() / count) < 1e-12 and rows[1] == 0
    dX, dW = S.distill_backward(X, W, ids, t, temperature, teacher_lse=tl, grad_loss=0.7)
    np.testing.assert_allclose(dX, tX.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(dW, tW.grad.numpy(), atol=1e-13)


def test_distillation_gradient_by_differences():
    X, W, ids, t = make(seed=5)
    dX, dW = S.distill_backward(X, W, ids, t, 1.7, "sum")
    h = 1e-6
    for at, A, d in (((2, 3), X, dX), ((4, 1), X, dX), ((7, 2), W, dW)):
        up, down = A.copy(), A.copy()
        up[at] += h
        down[at] -= h
        args = (lambda B: (B, W)) if A is X else (lambda B: (X, B))
        slope = (S.distill_forward(*args(up), ids, t, 1.7, "sum")[0]
                 - S.distill_forward(*args(down), ids, t, 1.7, "sum")[0]) / (2 * h)
        assert abs(slope - d[at]) < 1e-7


def test_distillation_from_the_student_itself_is_at_rest():
    """A teacher with the student's own logits on the whole vocabulary: no loss, no gradient."""
    X, W, _, _ = make()
    ids = np.tile(np.arange(11), (6, 1))
    loss, *_ = S.distill_forward(X, W, ids, X @ W.T, 1.3)
    dX, dW = S.distill_backward(X, W, ids, X @ W.T, 1.3)
    assert abs(loss) < 1e-14 and np.abs(dX).max() < 1e-14 and np.abs(dW).max() < 1e-14


def test_an_id_outside_the_vocabulary_or_no_entry_ignores_the_row():
    X, W, ids, t = make()
    ids[4, 1] = 11
    _, rows, _, logits, n = S.distill_forward(X, W, ids, t)
    dX, _ = S.distill_backward(X, W, ids, t)
    assert n == 4 and rows[4] == rows[1] == 0 and not dX[[1, 4]].any() and logits[4, 1] == 0
