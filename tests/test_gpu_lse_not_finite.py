"""Logits that are not finite in the losses' log-sum-exp: a NaN shows wherever it lies, and
columns of minus infinity weigh nothing."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
NAN = float("nan")


def make(N=70, H=64, V=3000, K=5, seed=31):
    import torch
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(N, H, generator=gen).bfloat16().cuda()
    X[:, 0] = 1.0
    W = (torch.randn(V, H, generator=gen) * 0.5 / H**0.5).bfloat16().cuda()
    # no label and no entry among the columns from 256 on up to 1024
    y = torch.randint(1024, V, (N, K), generator=gen).cuda()
    return X, W, y, torch.randn(N, K, generator=gen).cuda()


def losses(X, W, y, t):
    """(loss, rows' losses, lse) of the distillation, of the loss, and of the loss in two
    vocabulary shards."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    N, V = X.shape[0], W.shape[0]
    rows = torch.zeros(N, device="cuda")
    loss, lse, *_ = B.flce_distill_forward(X, W, y, t, row_loss=rows)
    yield loss, rows, lse
    labels, rows = y[:, 0].contiguous(), torch.zeros(N, device="cuda")
    loss, lse, *_ = B.flce_forward(X, W, labels, row_loss=rows)
    yield loss, rows, lse
    cut = 1024
    parts = [B.flce_forward_vocab_shard(X, W[a:b], labels, a, V)[0] for a, b in ((0, cut), (cut, V))]
    rows = torch.zeros(N, device="cuda")
    loss, lse, *_ = B.flce_combine_vocab_shards(torch.stack(parts), labels, V, B.make_options(row_loss=rows))
    yield loss, rows, lse


def test_a_token_of_nan():
    X, W, y, t = make()
    X[9, 7] = NAN
    keep = [i for i in range(70) if i != 9]
    for loss, rows, lse in losses(X, W, y, t):
        assert loss.isnan().all() and lse[9].isnan() and rows[9].isnan()
        assert lse[keep].isfinite().all() and rows[keep].isfinite().all()


@pytest.mark.parametrize("first,last", [(256, 512), (256, 1024), (0, 1024), (300, 301)])
def test_vocabulary_rows_of_nan(first, last):
    """One of them, a whole tile, several, a whole shard: no label and no entry among them."""
    X, W, y, t = make()
    W[first:last] = NAN
    for loss, rows, lse in losses(X, W, y, t):
        assert loss.isnan().all() and rows.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("first,last", [(256, 512), (0, 1024), (256, 320), (0, 64), (300, 301)])
def test_columns_of_minus_infinity(first, last):
    """They weigh nothing: lse is what the other columns give, within the rounding of sums of
    up to 3000 exponentials in two orders and of the tensor cores' products (2e-6 each of values
    below 10)."""
    import torch
    X, W, y, t = make()
    W[first:last] = 0
    W[first:last, 0] = -float("inf")
    z = X.double() @ torch.cat([W[:first], W[last:]]).double().T
    want = torch.logsumexp(z, -1)
    for loss, rows, lse in losses(X, W, y, t):
        assert loss.isfinite().all() and rows.isfinite().all()
        assert (lse.double() - want).abs().max() <= 4e-5
