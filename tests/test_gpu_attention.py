"""Packed causal attention against the fp64 oracle.

Tolerances, in relative Frobenius norm: out carries two roundings to bf16 (the
probabilities and the result), each of relative error 2^-9 / sqrt(3) = 1.1e-3
on average and 2^-8 together at most in the aligned case: 5e-3.  Gradients
carry up to four such roundings (out in delta, p, ds, the result): 1e-2, the
loss's own bar.  lse is fp32 throughout: 1e-4 absolute for scores up to ~50."""
import numpy as np
import pytest

from oracle import attn_oracle as A
from tests.gpu_util import rel_fro, tensor_f64

pytestmark = pytest.mark.gpu
OUT, GRAD, LSE = 5e-3, 1e-2, 1e-4


def make(T, HQ, HK, D, seed=0, spread=1.0, pad=0):
    """q, k, v as views of one buffer (with `pad` more values per head), and dout."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    buf = torch.randn(T, HQ + 2 * HK, D + pad, generator=gen)
    buf[:, :HQ] *= spread
    buf = buf.bfloat16().cuda()
    q, k, v = buf[:, :HQ, :D], buf[:, HQ:HQ + HK, :D], buf[:, HQ + HK:, :D]
    g = torch.randn(T, HQ, D, generator=gen).bfloat16().cuda()
    return q, k, v, g


def offsets(cu):
    import torch
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def run(q, k, v, g, cu, scale=None):
    from linear_cross_entropy_logit_gb300 import binding as B
    out, lse, err = B.flce_attention_forward(q, k, v, offsets(cu), scale)
    dq, dk, dv, _ = B.flce_attention_backward(g, q, k, v, out, lse, offsets(cu), scale,
                                              err_word=err)
    return out, lse, dq, dk, dv, int(err.item())


def check(q, k, v, g, cu, scale=None):
    got = run(q, k, v, g, cu, scale)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    qf, kf, vf, gf = (tensor_f64(t) for t in (q, k, v, g))
    out, lse = A.attention_forward(qf, kf, vf, cu, scale)
    grads = A.attention_backward(gf, qf, kf, vf, cu, scale)
    assert got[5] == 0
    assert rel_fro(tensor_f64(got[0]), out) <= OUT
    have = tensor_f64(got[1])
    assert (np.isneginf(have) == np.isneginf(lse)).all()
    live = np.isfinite(lse)
    assert np.abs(have[live] - lse[live]).max(initial=0.0) <= LSE
    for name, a, b in zip(("dq", "dk", "dv"), got[2:5], grads):
        # one visible key: the gradients of q and k are zero, what is left is rounding
        if np.linalg.norm(b) > 1e-9 * np.linalg.norm(gf):
            assert rel_fro(tensor_f64(a), b) <= GRAD, name
        else:
            assert np.abs(tensor_f64(a)).max(initial=0.0) <= 1e-2 * np.abs(gf).max(initial=0.0), name
    return got


LENGTHS = [[1], [2], [63], [64], [65], [127], [128], [129], [255], [256], [257], [300, 1, 0, 77],
           [0, 0, 5], [1, 1, 1, 1], [128, 128], [511, 513], [40] * 13]


@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "_".join(map(str, x[:4])))
@pytest.mark.parametrize("D", [64, 128])
def test_lengths(lengths, D):
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    check(*make(cu[-1], 4, 2, D, seed=len(lengths) + D), cu)


@pytest.mark.parametrize("D", [8, 16, 40, 72, 80, 96, 104, 120])
def test_head_sizes(D):
    check(*make(333, 2, 1, D, seed=D), [0, 100, 333])


@pytest.mark.parametrize("HQ,HK", [(1, 1), (3, 3), (7, 1), (8, 2), (32, 8), (14, 2)])
def test_head_groups(HQ, HK):
    check(*make(290, HQ, HK, 64, seed=HQ), [0, 150, 290])


@pytest.mark.parametrize("D", [64, 128])
def test_a_long_sequence(D):
    check(*make(1800, 4, 1, D, seed=1), [0, 1800])


def test_many_sequences():
    rng = np.random.default_rng(2)
    lengths = rng.integers(0, 9, 700)
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    check(*make(cu[-1] + 5, 2, 2, 64, seed=2), cu)


@pytest.mark.parametrize("D", [64, 128])
def test_many_units_for_each_sm(D):
    """Several ragged units, one after the other, on every CTA, beside rows that hold NaN."""
    lengths = [700, 130, 1, 0, 385, 64, 511, 257, 900, 33]
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    q, k, v, g = make(cu[-1] + 77, 32, 16, D, seed=D)
    for t in (q, k, v, g):
        t[cu[-1]:] = float("nan")
    got = run(q, k, v, g, cu)
    n = cu[-1]
    want = check(*[t[:n] for t in (q, k, v, g)], cu)
    import torch
    assert all(torch.equal(a[:n], b) for a, b in zip((got[0], *got[2:5]), (want[0], *want[2:5])))


def test_rows_outside_the_sequences():
    """Rows before the first and after the last sequence: out 0, lse -inf, gradients 0,
    whatever they hold."""
    import torch
    q, k, v, g = make(700, 4, 2, 128, seed=3)
    for t in (q, k, v, g):
        t[:130] = float("nan")
        t[601:] = float("inf")
    out, lse, dq, dk, dv, err = run(q, k, v, g, [130, 400, 601])
    assert err == 0
    for t in (out, dq, dk, dv):
        assert not t[:130].any() and not t[601:].any()
    assert torch.isneginf(lse[:, :130]).all() and torch.isneginf(lse[:, 601:]).all()
    inner = slice(130, 601)
    check_inner = [t[inner].clone() for t in (q, k, v, g)]
    want = run(*check_inner, [0, 270, 471])
    for a, b in zip((out, dq, dk, dv), (want[0], *want[2:5])):
        assert torch.isfinite(a[inner]).all() and torch.equal(a[inner], b)


def test_sequences_do_not_touch_each_other():
    """A sequence's results do not depend on what else is in the pack, bit for bit,
    even beside non-finite values."""
    import torch
    q, k, v, g = make(500, 4, 2, 64, seed=4)
    mid = slice(150, 333)
    alone = run(*[t[mid].clone() for t in (q, k, v, g)], [0, 183])
    for t in (q, k, v, g):
        t[:150] = float("nan")
        t[333:] = float("-inf")
    packed = run(q, k, v, g, [0, 150, 333, 500])
    for i in (0, 2, 3, 4):
        assert torch.equal(packed[i][mid], alone[i])
    assert torch.equal(packed[1][:, mid], alone[1])


@pytest.mark.parametrize("at", [5, 200])
def test_nonfinite_values_stay_out_of_masked_places(at):
    """A non-finite token reaches no earlier row: out and dq before it, and dk, dv after it,
    are what they are without it."""
    import torch
    for bad in (float("nan"), float("inf")):
        q, k, v, g = make(260, 2, 1, 64, seed=5)
        cu = [0, 260]
        clean = run(q, k, v, g, cu)
        v2 = v.clone()
        v2[at, 0, 3] = bad
        out, lse, *_ = run(q, k, v2, g, cu)
        assert torch.equal(out[:at], clean[0][:at]) and torch.equal(lse, clean[1])
        assert not torch.isfinite(out[at:, :, 3]).any()
        assert torch.equal(out[:, :, :3], clean[0][:, :, :3])
        k2 = k.clone()
        k2[at, 0, 3] = bad
        got = run(q, k2, v, g, cu)
        assert torch.equal(got[0][:at], clean[0][:at]) and torch.equal(got[2][:at], clean[2][:at])
        g2 = g.clone()
        g2[at, 0, 3] = bad
        got = run(q, k, v, g2, cu)
        assert torch.equal(got[3][at + 1:], clean[3][at + 1:])
        assert torch.equal(got[4][at + 1:], clean[4][at + 1:])


def test_large_scores():
    """Scores of several hundred: the running maximum keeps the exponentials in range."""
    q, k, v, g = make(400, 2, 1, 64, seed=6, spread=40.0)
    out, lse, dq, dk, dv, err = run(q, k, v, g, [0, 400])
    qf, kf, vf = (tensor_f64(t) for t in (q, k, v))
    want, wl = A.attention_forward(qf, kf, vf, [0, 400], 64 ** -0.5)
    assert err == 0 and rel_fro(tensor_f64(out), want) <= OUT
    # fp32 scores of up to ~200 carry an absolute error of ~200 * 2^-22
    assert np.abs(tensor_f64(lse) - wl).max() <= 1e-3


def test_falling_and_rising_scores():
    """Scores that rise or fall along the sequence by far more than one rescaling step."""
    for sign in (1.0, -1.0):
        q, k, v, g = make(1000, 1, 1, 64, seed=7)
        import torch
        ramp = torch.linspace(0, 30 * sign, 1000, device="cuda")[:, None]
        k = k.clone()
        k[:, :, 0] = ramp.bfloat16()
        q = q.clone()
        q[:, :, 0] = 8.0
        check(q, k, v, g, [0, 1000])


def test_strided_views_and_scale():
    q, k, v, g = make(310, 4, 2, 72, seed=8, pad=24)
    check(q, k, v, g, [0, 310], scale=0.31)
    # heads outermost in memory
    q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    check(q, k, v, g, [0, 17, 310])


def test_bad_offsets_are_reported():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, g = make(300, 2, 1, 64, seed=9)
    for cu in ([0, 200, 100, 300], [0, 301], [-1, 300]):
        out, lse, dq, dk, dv, err = run(q, k, v, g, cu)
        assert err == B.FLCE_ERR_INDEX
        assert torch.isneginf(lse).all() and not any(t.any() for t in (out, dq, dk, dv))


def test_no_tokens_and_no_sequences():
    import torch
    q, k, v, g = make(0, 2, 1, 64)
    assert run(q, k, v, g, [0])[5] == 0 and run(q, k, v, g, [0, 0])[5] == 0
    q, k, v, g = make(5, 2, 1, 64)
    out, lse, dq, dk, dv, err = run(q, k, v, g, [0])
    assert err == 0 and torch.isneginf(lse).all() and not any(t.any() for t in (out, dq, dk, dv))


def test_runs_give_the_same_bits():
    import torch
    q, k, v, g = make(2000, 8, 2, 128, seed=10)
    cu = [0, 700, 701, 1990]
    r = [run(q, k, v, g, cu) for _ in range(3)]
    for other in r[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r[0][:5], other[:5]))


def test_gradient_against_differences():
    """Directional derivatives of the 64-bit forward against the kernels' gradients."""
    q, k, v, g = make(90, 2, 1, 64, seed=11)
    cu, scale, h = [0, 40, 90], 0.125, 1e-5
    got = run(q, k, v, g, cu, scale)
    x = [tensor_f64(t) for t in (q, k, v)]
    gf = tensor_f64(g)
    rng = np.random.default_rng(12)
    for i in range(3):
        u = rng.standard_normal(x[i].shape)
        f = [float((A.attention_forward(*[x[j] + (s * h * u if j == i else 0.0) for j in range(3)],
                                        cu, scale)[0] * gf).sum()) for s in (1, -1)]
        have = tensor_f64(got[2 + i])
        # the gradient's error (GRAD of its norm) falls on the direction at random: u is a
        # unit normal per coordinate, so 4 standard deviations
        assert abs((f[0] - f[1]) / (2 * h) - float((have * u).sum())) <= 4 * GRAD * np.linalg.norm(have)


def test_autograd_graph_and_streams():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, g = make(300, 4, 2, 64, seed=13)
    cu = offsets([0, 120, 300])
    want = run(q, k, v, g, [0, 120, 300])
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = B.packed_attention(*leaves, cu)
        out.backward(g)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want[0])
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want[2:5]))
    # an explicit stream, then capture and replay
    o2, l2, _ = B.flce_attention_forward(q, k, v, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o2, want[0]) and torch.equal(l2, want[1])
    err = B.new_err_word("cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    grads = [torch.empty_like(w) for w in want[2:5]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.flce_attention_forward(q, k, v, cu, out=out, lse=lse, err_word=err)
        B.flce_attention_backward(g, q, k, v, out, lse, cu, dq=grads[0], dk=grads[1],
                                  dv=grads[2], err_word=err)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(a, b) for a, b in zip(grads, want[2:5]))


def test_debug_build_gives_the_same_bits():
    """The bounds-checked build finds no unit out of range and computes the same."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, g = make(777, 4, 2, 128, seed=14)
    cu = [3, 100, 100, 400, 770]
    want = run(q, k, v, g, cu)
    prev = B.use_library(B.load(B.DEBUG_LIB_PATH))
    try:
        got = run(q, k, v, g, cu)
    finally:
        B.use_library(prev)
    assert got[5] == 0 and all(torch.equal(a, b) for a, b in zip(want[:5], got[:5]))


# what the scores of a lower key tile's halves add to the diagonal tile's
JUMPS = [(0, 20), (20, 0), (300, 0), (0, 300), (100, 400), (400, 100), (-300, 60), (60, -300), (8, 8)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first,second", JUMPS)
def test_scores_that_jump_between_halves_of_a_tile(first, second, D):
    """The softmax's reference moves with either half of a key tile, at either of two tiles."""
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v, _ = make(400, 2, 1, D, seed=15)
    q[:, :, 0] = 1
    k[:, :, 0] = 0
    k[128:192, :, 0], k[192:256, :, 0] = first, second  # exact in bf16
    k[:64, :, 0], k[64:128, :, 0] = second, first
    out, lse, err = B.flce_attention_forward(q, k, v, offsets([0, 400]), 1.0)
    want, want_lse = A.attention_forward(*(tensor_f64(t) for t in (q, k, v)), [0, 400], 1.0)
    assert int(err.item()) == 0
    assert rel_fro(tensor_f64(out), want) <= OUT
    # LSE holds for scores up to 50; beyond, fp32's step grows with them
    bound = LSE * np.maximum(1.0, np.abs(want_lse) / 50)
    assert (np.abs(tensor_f64(lse) - want_lse) <= bound).all()


@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_minus_infinity_have_no_weight(D):
    """Scores of -infinity: in the diagonal tile of rows that see finite ones below it, and
    everywhere (those rows have no softmax)."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    for lo, hi in ((128, 400), (0, 200), (140, 150)):
        q, k, v, _ = make(400, 4, 2, D, seed=16)
        q[:, :, 0] = 1
        k[lo:hi, :, 0] = float("-inf")
        out, lse, err = B.flce_attention_forward(q, k, v, offsets([0, 400]))
        with np.errstate(invalid="ignore"):
            want, want_lse = A.attention_forward(*(tensor_f64(t) for t in (q, k, v)), [0, 400], D**-0.5)
        rows = np.arange(400)
        live = (rows < lo) | (rows >= hi) | (lo > 0)
        assert int(err.item()) == 0
        assert rel_fro(tensor_f64(out)[live], want[live]) <= OUT
        assert np.abs(tensor_f64(lse)[:, live] - want_lse[:, live]).max() <= LSE
        assert torch.isneginf(lse[:, torch.from_numpy(~live).cuda()]).all()


@pytest.mark.parametrize("D", [64, 80, 128])
def test_first_tokens_take_no_gradient_through_the_softmax(D):
    """A row with one visible key: dq is 0, and dk gets nothing from it (sequences of one
    token: all of dq and dk are 0, exactly; dv is dout, summed over the heads of a group)."""
    import torch
    q, k, v, g = make(190, 6, 2, D, seed=17, spread=4.0)
    cu = [0, 1, 2, 2, 3, 130, 131, 131, 185]
    _, _, dq, dk, dv, err = run(q, k, v, g, cu)
    starts = [a for a, b in zip(cu, cu[1:]) if b > a]
    ones = [a for a, b in zip(cu, cu[1:]) if b == a + 1]
    assert err == 0
    assert not dq[starts].any() and not dk[ones].any()
    want = g.float().view(190, 2, 3, D).sum(2).bfloat16()
    assert (dv[ones].float() - want[ones].float()).abs().max() <= 2.0**-7 * want.float().abs().max()
    # what the gradient holds that is not finite is not hidden by it
    g[0, 0, 0] = float("nan")
    _, _, dq, dk, _, _ = run(q, k, v, g, cu)
    assert torch.isnan(dq[0, 0]).all() and torch.isnan(dk[0, 0]).all() and not dq[1].any()
