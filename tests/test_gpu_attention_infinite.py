"""Packed attention with infinite and very large inputs against the fp64 oracle.

Tolerances as for ordinary inputs, over the values that the oracle has finite: OUT and GRAD
in relative Frobenius norm (two and up to four roundings to bf16).  Where the oracle has NaN
the kernels have to have NaN."""
import numpy as np
import pytest

from oracle import attn_oracle as A
from tests.gpu_util import tensor_f64
from tests.test_gpu_attention import GRAD, LSE, OUT, make, run

pytestmark = pytest.mark.gpu


def oracle(q, k, v, g, cu, scale=None):
    """(out, dq, dk, dv) in 64 bits."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q, k, v, g = (tensor_f64(t) for t in (q, k, v, g))
    with np.errstate(invalid="ignore"):
        return (A.attention_forward(q, k, v, cu, scale)[0], *A.attention_backward(g, q, k, v, cu, scale))


def close(got, want, bound, name):
    """NaN where the oracle has NaN; the other values within `bound` of its norm."""
    got = tensor_f64(got)
    assert (np.isnan(got) == np.isnan(want)).all(), name
    live = np.isfinite(want)
    assert np.linalg.norm(got[live] - want[live]) <= bound * np.linalg.norm(want[live]), name


# tokens and the infinite keys: within a sequence's first 128 rows alone, in a later diagonal
# tile, in both; a last tile that is full and one that is not
WEIGHTLESS = [(100, [40]), (128, [1, 127]), (300, [200]), (300, [3, 130, 299]), (384, [150, 383]),
              (700, [90, 300, 301, 650])]


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("tokens,bad", WEIGHTLESS, ids=lambda x: str(x))
@pytest.mark.parametrize("value", [float("-inf"), float("inf")])
def test_gradients_beside_keys_without_weight(tokens, bad, D, value):
    """Keys whose scores are all -infinity: they have no weight, so that the other keys'
    gradients and the finite components of dq are the oracle's; dq is NaN (0 x infinity) in the
    infinite component of the rows that see one."""
    q, k, v, g = make(tokens + 40, 4, 2, D, seed=tokens + D)
    q[:, :, 0] = 1.0 if value < 0 else -1.0
    k[bad, :, 0] = value
    cu = [0, tokens, tokens + 40]
    _, _, dq, dk, dv, err = run(q, k, v, g, cu)
    _, want_q, want_k, want_v = oracle(q, k, v, g, cu)
    # the oracle multiplies masked keys by zero: rows before the first infinite one by themselves
    n = bad[0]
    want_q[:n] = oracle(q[:n], k[:n], v[:n], g[:n], [0, n])[1]
    assert err == 0
    close(dq, want_q, GRAD, "dq")
    others = np.setdiff1d(np.arange(tokens + 40), bad)
    close(dk[others], want_k[others], GRAD, "dk")
    close(dv[others], want_v[others], GRAD, "dv")


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("tokens,bad", WEIGHTLESS, ids=lambda x: str(x))
def test_keys_without_weight_get_no_gradient(tokens, bad, D):
    """dk and dv of a key whose scores are all -infinity are 0, whatever the length leaves empty
    in the last tile of queries."""
    q, k, v, g = make(tokens, 4, 2, D, seed=tokens + D)
    q[:, :, 0] = 1.0
    k[bad, :, 0] = float("-inf")
    _, _, _, dk, dv, err = run(q, k, v, g, [0, tokens])
    assert err == 0
    assert (dk[bad] == 0).all() and (dv[bad] == 0).all()


BF16_MAX = 3.3895313892515355e38


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [1, 70, 300, 1100])
@pytest.mark.parametrize("size", [1e30, 5e36, 0.99 * BF16_MAX])
def test_large_values_stay_finite(size, tokens, D):
    """Finite values give finite results: neither the number of keys nor scores that rise above
    the softmax's reference by less than what moves it take a sum past fp32."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, _ = make(tokens, 2, 1, D, seed=18)
    v = (torch.rand(tokens, 1, D, generator=torch.Generator().manual_seed(19)) * 0.5 + 0.49).cuda()
    v = (v * size).bfloat16()
    cu = [0, tokens]
    for rise in (0.0, 10.0):  # of the scores from the diagonal tile to the first key: 10 < 16 ln 2
        q, k = q * 0, k * 0
        q[:, :, 0] = 1.0
        k[:, 0, 0] = torch.linspace(rise, 0, tokens)
        out, lse, err = B.flce_attention_forward(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 1.0)
        want, want_lse = A.attention_forward(*(tensor_f64(t) for t in (q, k, v)), cu, 1.0)
        assert int(err.item()) == 0
        close(out, want, OUT, "out")
        assert np.abs(tensor_f64(lse) - want_lse).max() <= LSE


@pytest.mark.parametrize("D", [64, 128])
def test_small_values_keep_their_accuracy(D):
    """The same at the other end: values of 1e-30 are not lost."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, _ = make(500, 2, 1, D, seed=20)
    v = (v.float() * 1e-30).bfloat16()
    cu = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    out, _, err = B.flce_attention_forward(q, k, v, cu)
    want, _ = A.attention_forward(*(tensor_f64(t) for t in (q, k, v)), [0, 500], D ** -0.5)
    assert int(err.item()) == 0
    close(out, want, OUT, "out")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [7, 200])
def test_a_query_without_softmax_reaches_the_keys_it_sees(at, D):
    """A row whose scores are all -infinity has no softmax: its dq, and dk and dv of the keys it
    sees, are NaN, in the diagonal tile as in the others."""
    import torch
    q, k, v, g = make(300, 2, 2, D, seed=21)
    q[at, :, 0] = float("-inf")
    k[:, :, 0] = 1.0
    _, lse, dq, dk, dv, err = run(q, k, v, g, [0, 300])
    assert err == 0 and torch.isneginf(lse[:, at]).all()
    assert torch.isnan(dq[at]).all()
    for t in (dk, dv):
        assert torch.isnan(t[:at + 1]).all() and torch.isfinite(t[at + 1:]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_from_zero(sign, D):
    """Scores of 2^24 in size and one step nearer to zero (both exact in fp32): every row, the first
    as well, has a finite softmax."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, _ = make(300, 2, 1, D, seed=23)
    q, k = q * 0, k * 0
    q[:, :, 0], q[:, :, 1] = 4096, 1
    k[:, :, 0] = 4096 * sign
    k[::3, :, 1] = -sign
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    out, lse, err = B.flce_attention_forward(q, k, v, cu, 1.0)
    want, want_lse = A.attention_forward(*(tensor_f64(t) for t in (q, k, v)), [0, 300], 1.0)
    assert int(err.item()) == 0
    # a score times log2 e is rounded in fp32 once (the fused multiply-add's own result is small)
    close(out, want, OUT, "out")
    assert np.abs(tensor_f64(lse) - want_lse).max() <= 2.0**-22 * 2.0**24


def by_pairs(q, k, v, g, cu, scale):
    """(out, dq, dk, dv) in 64 bits from the visible pairs alone, row by row: a masked pair is not
    even multiplied by zero."""
    group = q.shape[1] // k.shape[1]
    out, dq, dk, dv = (np.zeros_like(t) for t in (q, q, k, v))
    for lo, hi in zip(cu, cu[1:]):
        for h in range(q.shape[1]):
            kh = h // group
            for i in range(lo, hi):
                seen = slice(lo, i + 1)
                s = scale * (k[seen, kh] @ q[i, h])
                e = np.exp(s - s.max())
                p = e / e.sum()
                dp = v[seen, kh] @ g[i, h]
                ds = p * (dp - (p * dp).sum())
                out[i, h] = p @ v[seen, kh]
                dq[i, h] = scale * (ds @ k[seen, kh])
                dk[seen, kh] += scale * np.outer(ds, q[i, h])
                dv[seen, kh] += np.outer(p, g[i, h])
    return out, dq, dk, dv


@pytest.mark.parametrize("seed", range(24))
def test_random_places_that_are_not_finite(seed):
    """Infinities and NaN anywhere in one of q, k, v and dout: the results are finite exactly where
    the formulas' are, and right there."""
    rng = np.random.default_rng(seed)
    D, HK = int(rng.choice([8, 64, 72, 128])), int(rng.choice([1, 2]))
    HQ = HK * int(rng.choice([1, 2, 3]))
    cu = np.cumsum([0, *rng.choice([1, 5, 64, 100, 128, 129, 200, 257], int(rng.integers(1, 4)))]).tolist()
    x = list(make(cu[-1], HQ, HK, D, seed=seed))
    if rng.integers(2):  # infinite keys then have scores of one sign
        x[0] = x[0].abs()
    t = x[seed % 4]
    for _ in range(int(rng.integers(1, 4))):
        t[tuple(int(rng.integers(n)) for n in t.shape)] = float(rng.choice([np.inf, -np.inf, -np.inf, np.nan]))
    out, _, dq, dk, dv, err = run(*x, cu)
    assert err == 0
    with np.errstate(all="ignore"):
        want = by_pairs(*(tensor_f64(t) for t in x), cu, D ** -0.5)
    for name, a, b, bound in zip(("out", "dq", "dk", "dv"), (out, dq, dk, dv), want, (OUT, GRAD, GRAD, GRAD)):
        a, live = tensor_f64(a), np.isfinite(b)
        assert (np.isfinite(a) == live).all(), name
        # short sequences alone have next to no gradient of q and k: what is left is rounding of dout's size
        size = max(np.linalg.norm(b[live]), 0.1)
        assert np.linalg.norm(a[live] - b[live]) <= bound * size, name
