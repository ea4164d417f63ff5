"""Linear distillation where exponentials underflow, overflow or lose their digits.  Tolerances
as in test_gpu_distill."""
import pytest

from tests.test_gpu_distill import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _defaults():
    from linear_cross_entropy_logit_gb300 import binding as B
    yield
    B.flce_set_vocab_chunk(0)


FAR = [95.0, 200.0, 1e4, float("inf")]  # above the entries: probabilities of 1e-42, then zeros


@pytest.mark.parametrize("chunk", [0, 512])
@pytest.mark.parametrize("grad", [1.0, -2.0])
@pytest.mark.parametrize("where", ["some", "all"])
def test_entries_far_below_the_teachers_sum(where, grad, chunk):
    """Rows whose entries all have probability 0 count, have no loss and no gradient, and leave
    the others' alone."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    B.flce_set_vocab_chunk(chunk)
    X, W, ids, t = make(300, 128, 3001, 9, seed=21)
    T = 1.5
    tl = torch.logsumexp(t / T, -1).nan_to_num(0.0, neginf=0.0) + 0.2
    if where == "some":
        for i, far in enumerate(FAR):
            tl[[10 + i, 100 + i, 296 + i]] += far
    else:
        tl += 200.0
        tl[::5] = float("inf")
    rows = torch.full((300,), float("nan"), device="cuda")
    B.flce_distill_forward(X, W, ids, t, T, teacher_lse=tl, row_loss=rows)
    out, grads, err = run(B, X, W, ids, t, T, "mean", tl, torch.tensor([grad], device="cuda"))
    assert int(err.item()) == 0 and not rows[tl > 150.0].any()
    assert not grads[0][tl > 150.0].any()
    if where == "all":
        # every q is at most exp(-200) = 1e-87, so the formulas' loss and gradients are below 1e-80
        # and their float nearest is 0 (the smallest is 1e-45)
        assert not out[0].any() and int(out[3].item()) == 298 and not grads[0].any() and not grads[1].any()
    else:
        check(X, W, ids, t, T, tl, "mean", out, grads, grad)


@pytest.mark.parametrize("pattern", ["end", "between"])
@pytest.mark.parametrize("grad", [-2.0, 2.0])
def test_large_logits_of_tokens_that_do_not_count(grad, pattern):
    """Their z / T pass what an exponential holds, 88; with either sign of the upstream
    gradient they leave no trace."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(150, 64, 700, 6, seed=22, odd_rows=False)
    at = torch.arange(150, device="cuda")
    out_of = at >= 80 if pattern == "end" else at % 15 < 7
    assert int(out_of.sum()) == 70
    ids[out_of] = -1
    T = 0.01
    assert float((X.float() @ W.float().T / T)[out_of].amax(-1).min()) > 89.0
    out, (dX, dW), err = run(B, X, W, ids, t, T, grad=torch.tensor([grad], device="cuda"))
    assert int(err.item()) == 0 and not dX[out_of].any()
    check(X, W, ids, t, T, None, "mean", out, (dX, dW), grad)
