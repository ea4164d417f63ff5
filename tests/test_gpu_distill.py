"""Linear distillation against the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-24):
  logits   a sum of H exact products over lanes of H / 32: (H / 32 + 8) u of the sum of
           their magnitudes
  lse      logits of the tensor cores: H / 16 steps, each off by at most 2 u of the sum of
           magnitudes so far; the exponentials' and the sums' roundings, 2e-6
  loss     sum of q times the logits' error over T, plus lse's
  dZ       its rounding to bf16, 2^-8 of each value; before that, p's relative error, which is
           lse's error plus the logits', of p (not of p - q)
  dX, dW   that, through the products; their own rounding to bf16, 2^-8; by value these bounds
           are far above what independent roundings add up to, so also in norm: two roundings
           of 2^-9 / sqrt(3) each are 1.6e-3, 4e-3 leaves room for dZ that is uneven."""
import numpy as np
import pytest

from oracle import step_oracle as S
from tests.gpu_util import rel_fro, tensor_f64

pytestmark = pytest.mark.gpu
U = 2.0**-24


@pytest.fixture(autouse=True)
def _defaults():
    from linear_cross_entropy_logit_gb300 import binding as B
    yield
    B.flce_set_vocab_chunk(0)
    B.flce_set_cluster_multicast(True)


def make(N, H, V, K, dtype="fp32", seed=0, odd_rows=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(N, H, generator=gen).bfloat16()
    W = (torch.randn(V, H, generator=gen) * 0.5 / H**0.5).bfloat16()
    ids = torch.stack([torch.randperm(V, generator=gen)[:K] for _ in range(N)]) if N else torch.zeros(0, K).long()
    t = 2 * torch.randn(N, K, generator=gen)
    if odd_rows and N > 6:
        ids[1] = -1                # no entry
        ids[2, K // 2:] = -100     # fewer
        t[3] = -float("inf")       # entries without weight
        t[4, 0] = -float("inf")
        ids[5, K - 1] = ids[5, 0]  # the same id twice (with K = 1 once)
    t = t.to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype])
    return X.cuda(), W.cuda(), ids.cuda(), t.cuda()


def check(X, W, ids, t, T, tl, reduction, out, grads, grad=1.0):
    """The call's results against the oracle's, by the bounds above."""
    loss, lse, logits, valid = out
    x, w, i, tt = tensor_f64(X), tensor_f64(W), ids.cpu().numpy(), tensor_f64(t)
    N, H = x.shape
    tail = None if tl is None else tensor_f64(tl)
    wl, rows, wlse, wz, n = S.distill_forward(x, w, i, tt, T, reduction, tail)
    q, _, ok = S.teacher(i, tt, T, len(w), tail)
    size = np.abs(x) @ np.abs(w).T
    known = (i >= 0) & (i < len(w))
    zerr = (H / 32 + 8) * U * np.where(known, np.take_along_axis(size, np.where(known, i, 0), 1), 0.0)
    assert int(valid) == n
    assert (np.abs(tensor_f64(logits) - wz) <= zerr).all()
    lerr = (H / 16 + 4) * 2 * U * size.max(-1, initial=0.0) / T + 2e-6 + 4 * U * np.abs(wlse)
    assert (np.abs(tensor_f64(lse) - wlse) <= lerr).all()
    # q, t and the logits divided by T in fp32: 4 u of each term
    terms = (q * (np.abs(wz / T) + np.where(np.isfinite(tt), np.abs(tt / T), 0.0))).sum(-1) + q.sum(-1) * np.abs(wlse)
    rerr = (q * zerr).sum(-1) / T + q.sum(-1) * lerr + 16 * U * terms
    assert abs(float(loss) - wl) <= rerr.sum() / (max(n, 1) if reduction == "mean" else 1) + U * abs(wl)
    if grads is None:
        return
    dX, dW = grads
    wx, ww = S.distill_backward(x, w, i, tt, T, reduction, tail, grad)
    p = np.exp(x @ w.T / T - wlse[:, None]) * (q.sum(-1) * ok)[:, None]
    d = p.copy()
    np.subtract.at(d, (np.nonzero(q)[0], i[np.nonzero(q)]), q[np.nonzero(q)])
    c = abs(grad) / T / (max(n, 1) if reduction == "mean" else 1)
    perr = (lerr + zerr.max(-1, initial=0.0) / T + 8 * U)[:, None]
    derr = c * (2.0**-8 * np.abs(d) + perr * p)
    acc = c * (np.abs(d) + p * perr)
    assert (np.abs(tensor_f64(dX) - wx) <= derr @ np.abs(w) * 1.01 + 2.0**-8 * np.abs(wx)
            + (len(w) / 16 + 8) * 2 * U * (acc @ np.abs(w)) + 1e-37).all()
    assert (np.abs(tensor_f64(dW) - ww) <= derr.T @ np.abs(x) * 1.01 + 2.0**-8 * np.abs(ww)
            + (N / 16 + 8) * 2 * U * (acc.T @ np.abs(x)) + 1e-37).all()
    if n and len(w) > 1:
        assert rel_fro(tensor_f64(dX), wx) <= 4e-3 and rel_fro(tensor_f64(dW), ww) <= 4e-3


def run(B, X, W, ids, t, T=1.0, reduction="mean", tl=None, grad=None, **kw):
    """Forward and backward, with workspaces and outputs full of NaN."""
    import torch
    (N, H), V, K = X.shape, W.shape[0], ids.shape[1]

    def workspace(mode):
        return torch.full((B.flce_distill_workspace_size(N, H, V, K, mode),), 255, dtype=torch.uint8, device="cuda")

    def junk(*shape, dtype=torch.float32):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    *out, err = B.flce_distill_forward(X, W, ids, t, T, reduction, teacher_lse=tl, loss=junk(1), lse=junk(N),
                                       logits=junk(N, K), workspace_buf=workspace(B.MODE_FWD))
    kw.setdefault("dW", junk(V, H, dtype=torch.bfloat16))
    dX, dW, _ = B.flce_distill_backward(X, W, ids, t, *out[1:], T, reduction, teacher_lse=tl, grad_loss=grad,
                                        err_word=err, dX=junk(N, H, dtype=torch.bfloat16),
                                        workspace_buf=workspace(B.MODE_BWD), **kw)
    return out, (dX, dW), err


CASES = [  # N, H, V, K, T, teacher's type, tail, reduction, chunk
    (1, 8, 8, 1, 1.0, "fp32", False, "mean", 0),
    (1, 4096, 1000, 64, 1.0, "bf16", False, "mean", 0),
    (7, 64, 257, 3, 2.0, "fp32", True, "sum", 0),
    (33, 136, 1031, 33, 0.5, "bf16", True, "mean", 256),
    (129, 72, 300, 300, 1.0, "fp32", False, "mean", 0),
    (255, 256, 4099, 16, 1.5, "fp32", False, "mean", 512),
    (300, 40, 5000, 100, 4.0, "bf16", True, "sum", 1024),
    (700, 1024, 3001, 50, 1.0, "fp32", False, "mean", 768),
    (1030, 264, 8000, 64, 1.3, "bf16", False, "mean", 2048),
    (20, 64, 2000, 1024, 1.0, "fp32", False, "mean", 0),
    # dX in parts of the contraction: 204 and 108 k-blocks, which 25 and 13 parts
    # would not divide
    (20, 64, 26200, 4, 1.0, "fp32", False, "mean", 13056),
    (90, 520, 14000, 4, 1.0, "fp32", False, "mean", 6912),
]


@pytest.mark.parametrize("N,H,V,K,T,dtype,tail,reduction,chunk", CASES)
def test_forward_and_backward(N, H, V, K, T, dtype, tail, reduction, chunk):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    B.flce_set_vocab_chunk(chunk)
    X, W, ids, t = make(N, H, V, K, dtype, seed=N + V)
    tl = (torch.rand(N, generator=torch.Generator().manual_seed(9)) + 5.0 / T).cuda() if tail else None
    grad = torch.tensor([0.75], device="cuda")
    out, grads, err = run(B, X, W, ids, t, T, reduction, tl, grad)
    assert int(err.item()) == 0
    check(X, W, ids, t, T, tl, reduction, out, grads, 0.75)


@pytest.mark.parametrize("multicast", [True, False])
def test_several_row_blocks_with_and_without_multicast(multicast):
    from linear_cross_entropy_logit_gb300 import binding as B
    B.flce_set_cluster_multicast(multicast)
    B.flce_set_vocab_chunk(4096)
    X, W, ids, t = make(1024, 128, 20000, 20, seed=3)
    out, grads, err = run(B, X, W, ids, t, 1.1)
    assert (B.last_multicast_launches() > 0) == multicast and int(err.item()) == 0
    check(X, W, ids, t, 1.1, None, "mean", out, grads)


@pytest.mark.parametrize("pattern", ["one", "last", "prompts", "half", "most", "three_blocks"])
@pytest.mark.parametrize("N", [1024, 1100])
def test_rows_that_do_not_count_lie_anywhere(N, pattern):
    """One row that counts, the last ones, all but prompts, every second, all but a few; an odd
    number of row blocks where they are walked in twos."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    B.flce_set_vocab_chunk(2048)
    X, W, ids, t = make(N, 128, 6000, 7, seed=N, odd_rows=False)
    at = torch.arange(N)
    counts = {"one": at == 777, "last": at >= N - 65, "prompts": at % 300 >= 140, "half": at % 2 == 0,
              "most": at % 97 != 5, "three_blocks": at % 16 < 11}[pattern]
    ids[~counts.cuda()] = -1
    out, (dX, dW), err = run(B, X, W, ids, t, 1.4)
    assert int(err.item()) == 0 and int(out[3].item()) == int(counts.sum())
    check(X, W, ids, t, 1.4, None, "mean", out, (dX, dW))
    assert not dX[~counts.cuda()].any()


def test_one_row_of_loss_each():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(70, 64, 500, 9, seed=4)
    rows = torch.full((70,), -1.0, device="cuda")
    B.flce_distill_forward(X, W, ids, t, 2.0, row_loss=rows)
    _, want, *_ = S.distill_forward(tensor_f64(X), tensor_f64(W), ids.cpu().numpy(), tensor_f64(t), 2.0)
    # terms below 10 in size, with fewer than 10 fp32 roundings each
    assert np.abs(tensor_f64(rows) - want).max() <= 100 * 2 * U * 10 and rows[1] == rows[3] == 0


def test_a_student_near_its_teacher_keeps_the_difference():
    """The teacher's entries are the student's own logits on the whole vocabulary: p - q is
    what fp32 leaves of it, 2e-5 of p, not bf16's rounding of p (2e-3)."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, _, _ = make(64, 256, 512, 1, seed=5)
    ids = torch.arange(512, device="cuda").repeat(64, 1)
    t = (X.double() @ W.double().T).float()
    out, (dX, dW), _ = run(B, X, W, ids, t)
    p = torch.softmax(X.double() @ W.double().T, -1) / 64
    assert abs(out[0].item()) <= 1e-5
    assert (dX.double().abs() <= 2e-5 * (p @ W.double().abs())).all()
    assert (dW.double().abs() <= 2e-5 * (p.T @ X.double().abs())).all()


def test_ids_outside_the_vocabulary_are_reported_and_their_rows_ignored():
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(40, 64, 300, 5, seed=6)
    ids[7, 2], ids[20, 4], ids[21, 0] = 300, 2**40, 2**31 + 5
    out, grads, err = run(B, X, W, ids, t)
    assert int(err.item()) == B.FLCE_ERR_LABEL
    check(X, W, ids, t, 1.0, None, "mean", out, grads)
    assert not grads[0][[1, 3, 7, 20, 21]].any() and int(out[3].item()) == 35


def test_no_row_counts_and_no_tokens():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(30, 64, 300, 5, seed=7)
    ids.fill_(-1)
    out, (dX, dW), err = run(B, X, W, ids, t, dW=torch.full((300, 64), 3.0, device="cuda").bfloat16())
    assert out[0].item() == 0 and out[3].item() == 0 and not dX.any() and not dW.any() and err.item() == 0
    for kw in ({}, {"dW": torch.full((300, 64), 3.0, device="cuda")}):
        out, (dX, dW), err = run(B, X[:0], W, ids[:0], t[:0], **kw)
        assert out[0].item() == 0 and out[3].item() == 0 and dX.shape == (0, 64) and not dW.any()
    acc = torch.full((300, 64), 3.0, device="cuda")
    run(B, X[:0], W, ids[:0], t[:0], dW=acc, accumulate_dW=True)
    assert (acc == 3.0).all()


def test_dw_in_fp32_accumulates_and_rounds_to_the_other():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    B.flce_set_vocab_chunk(512)
    X, W, ids, t = make(300, 128, 2000, 12, seed=8)
    _, (_, dW), _ = run(B, X, W, ids, t)
    _, (_, full), _ = run(B, X, W, ids, t, dW=torch.empty(2000, 128, device="cuda"))
    assert dW.dtype == torch.bfloat16 and full.dtype == torch.float32 and torch.equal(full.bfloat16(), dW)
    acc = torch.randn(2000, 128, device="cuda")
    want = acc + full
    run(B, X, W, ids, t, dW=acc, accumulate_dW=True)
    assert torch.equal(acc, want)


def test_what_is_not_finite_stays_in_its_row():
    """A NaN logit of the teacher makes its row's loss and gradient NaN, and of dW no more
    than the formula says (all of it: the row has a probability everywhere)."""
    from linear_cross_entropy_logit_gb300 import binding as B
    import torch
    X, W, ids, t = make(40, 64, 300, 5, seed=9)
    rows = torch.zeros(40, device="cuda")
    good, (gX, _), _ = run(B, X, W, ids, t, reduction="sum")
    t[9, 2], t[11, 0] = float("nan"), float("inf")
    B.flce_distill_forward(X, W, ids, t, row_loss=rows)
    _, (dX, _), err = run(B, X, W, ids, t, reduction="sum")
    keep = [i for i in range(40) if i not in (9, 11)]
    assert rows[[9, 11]].isnan().all() and rows[keep].isfinite().all() and int(err.item()) == 0
    assert dX[[9, 11]].isnan().all() and torch.equal(dX[keep], gX[keep])


def test_same_bits_on_other_streams_and_in_a_graph():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(520, 256, 6000, 30, seed=10)
    ws = torch.empty(B.flce_distill_workspace_size(520, 256, 6000, 30), dtype=torch.uint8, device="cuda")
    err = B.new_err_word("cuda")

    def step():
        *out, _ = B.flce_distill_forward(X, W, ids, t, 1.7, workspace_buf=ws, err_word=err)
        return *out, *B.flce_distill_backward(X, W, ids, t, *out[1:], 1.7, workspace_buf=ws, err_word=err)[:2]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(2):
        X.copy_(torch.roll(X, 1, 0))
        t.add_(0.5 * torch.randn_like(t))
        ids[k] = -1
        graph.replay()
        got = [o.clone() for o in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and err.item() == 0


def test_autograd():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(48, 64, 700, 6, seed=11)
    h, w = X.view(4, 12, 64).clone().requires_grad_(), W.clone().requires_grad_()
    err = B.new_err_word("cuda")
    loss = B.linear_distillation(h, w, ids.view(4, 12, 6), t.view(4, 12, 6), 2.0, err_word=err)
    (4.0 * loss).backward()
    out, grads, _ = run(B, X, W, ids, t, 2.0, grad=torch.tensor([4.0], device="cuda"))
    assert torch.equal(loss.detach(), out[0][0]) and err.item() == 0
    assert torch.equal(h.grad.view(48, 64), grads[0]) and torch.equal(w.grad, grads[1])
    check(X, W, ids, t, 2.0, None, "mean", out, grads, 4.0)


@pytest.mark.parametrize("N,H,V", [(300, 128, 2000), (20, 64, 30000)])
def test_a_gradient_that_is_not_needed_is_left_out(N, H, V):
    """Of frozen hidden states or a frozen matrix; the other one has the same bits."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(N, H, V, 8, seed=17)
    *out, err = B.flce_distill_forward(X, W, ids, t)
    dX, dW, _ = B.flce_distill_backward(X, W, ids, t, *out[1:])
    launches = B.last_launch_count()
    a, none, _ = B.flce_distill_backward(X, W, ids, t, *out[1:], need_dW=False)
    assert none is None and torch.equal(a, dX) and B.last_launch_count() < launches
    none, b, _ = B.flce_distill_backward(X, W, ids, t, *out[1:], need_dX=False)
    assert none is None and torch.equal(b, dW) and B.last_launch_count() < launches
    h = X.clone().requires_grad_()
    B.linear_distillation(h, W, ids, t).backward()
    assert torch.equal(h.grad, dX) and W.grad is None
    w = W.clone().requires_grad_()
    B.linear_distillation(X, w, ids, t).backward()
    assert torch.equal(w.grad, dW)


def test_gradient_by_differences():
    """The loss moves along a direction as the gradient says: with bf16 hidden states a step
    of one unit in the last place of every value, 2^-8 of them, of a fp64 loss."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(64, 128, 400, 8, seed=12, odd_rows=False)
    _, (dX, _), _ = run(B, X, W, ids, t, 1.5, "sum")
    step = (X.float() * 2.0**-6 * torch.randn(64, 128, generator=torch.Generator().manual_seed(1)).sign().cuda())
    up, down = (X.float() + step).bfloat16(), (X.float() - step).bfloat16()
    f = [S.distill_forward(tensor_f64(a), tensor_f64(W), ids.cpu().numpy(), tensor_f64(t), 1.5, "sum")[0]
         for a in (up, down)]
    along = float((dX.double() * (up.double() - down.double())).sum())
    # the gradient's error, 4e-3 of its norm at most, and the third order of the step
    assert abs(f[0] - f[1] - along) <= 4e-3 * float(dX.double().norm() * (up.double() - down.double()).norm())


@pytest.mark.parametrize("grad", [-2.0, 0.0, 1e-30])
def test_any_upstream_gradient(grad):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(150, 64, 700, 6, seed=14)
    out, (dX, dW), _ = run(B, X, W, ids, t, grad=torch.tensor([grad], device="cuda"))
    if grad == 0.0:
        assert not dX.any() and not dW.any()
    elif grad == 1e-30:  # dX is tiny, not zero: bf16 has fp32's exponents
        _, (one, _), _ = run(B, X, W, ids, t)
        assert rel_fro(tensor_f64(dX) / 1e-30, tensor_f64(one)) <= 4e-3
    else:
        check(X, W, ids, t, 1.0, None, "mean", out, (dX, dW), grad)


def test_calls_on_two_streams_at_once():
    """Each with its own workspace: the results of calls made alone."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    inputs = [make(600, 256, 9000, 24, seed=s) for s in (15, 16)]
    want = [run(B, *a, T=1.2)[:2] for a in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for a, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(run(B, *a, T=1.2))
        torch.cuda.synchronize()
        for (o, g, err), (wo, wg) in zip(got, want):
            assert int(err.item()) == 0 and all(torch.equal(a, b) for a, b in zip((*o, *g), (*wo, *wg)))


def test_debug_library():
    from linear_cross_entropy_logit_gb300 import binding as B
    X, W, ids, t = make(300, 136, 1500, 21, seed=13)
    want, grads, _ = run(B, X, W, ids, t)
    prev = B.use_library(B.load(B.DEBUG_LIB_PATH))
    try:
        got, other, err = run(B, X, W, ids, t)
    finally:
        B.use_library(prev)
    assert int(err.item()) == 0
    for a, b in zip((*want, *grads), (*got, *other)):
        assert (a == b).all()
