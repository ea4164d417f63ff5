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


def test_a_teachers_logits_may_lie_anywhere():
    """Probabilities go by differences: logits moved together by a number that moves them
    exactly give the same bits."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(130, 64, 700, 12, seed=23)
    t = (t * 8).round() / 8
    for T in (1.0, 0.7):
        want = run(B, X, W, ids, t, T)
        check(X, W, ids, t, T, None, "mean", *want[:2])
        for by in (2.0**19, -(2.0**19)):
            moved = t + by
            assert torch.equal(moved - by, t)
            got = run(B, X, W, ids, moved, T)
            for a, b in zip((*want[0], *want[1]), (*got[0], *got[1])):
                assert torch.equal(a, b)


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_entries_of_the_types_lowest_value(dtype, T):
    """They are entries, without weight next to any other; a row that has nothing else has them
    all alike."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(90, 64, 700, 12, dtype, seed=24, odd_rows=False)
    lowest = torch.finfo(t.dtype).min
    low, masked = t.clone(), t.clone()
    low[::3, 4:], masked[::3, 4:] = lowest, -float("inf")
    low[1::9], masked[1::9] = lowest, 0.0
    low[2::9, 1:], masked[2::9, 1:] = lowest, -float("inf")  # as far apart as the type goes
    low[2::9, 0], masked[2::9, 0] = -lowest, 0.0
    out, grads, err = run(B, X, W, ids, low, T)
    assert int(err.item()) == 0 and int(out[3].item()) == 90
    check(X, W, ids, masked, T, None, "mean", out, grads)
    # against the teacher's own sum they weigh nothing, and the row counts
    tl = torch.logsumexp(masked.float() / T, -1) + 0.1
    low[2::9, 0] = 0.0
    out, grads, _ = run(B, X, W, ids, low, T, tl=tl)
    assert int(out[3].item()) == 90 and not grads[0][1::9].any()
    check(X, W, ids, low, T, tl, "mean", out, grads)
