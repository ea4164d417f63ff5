"""Layer norm and RMS norm, forward and backward, against the fp64 oracle.

Tolerances: all arithmetic is fp32.  A row's sums run over at most 32 values a thread, then
over a tree of 10 levels: 42 roundings of 2^-24, 2.5e-6 of a sum of magnitudes, which for
these inputs is at most 4 times what it adds up to: 1e-5.  A bf16 output adds one rounding
to nearest, at most 2^-8 of its own value."""
import numpy as np
import pytest

from oracle import step_oracle as S
from tests.gpu_util import rel_fro, tensor_f64

pytestmark = pytest.mark.gpu
TOL = 1e-5
EPS = 1e-5


def near(got, want, dtype, tol=TOL):
    err = np.abs(tensor_f64(got) - want)
    if dtype == "bf16":
        err = np.maximum(0.0, err - 2.0**-8 * np.abs(want))
    return np.linalg.norm(err) <= tol * np.linalg.norm(want)


def make(R, H, dtype, seed=0, pad=0):
    """x and residual as views of wider rows, weight, bias, dy, ds."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (r(R, H + pad) * (0.5 + 3 * torch.rand(R, 1, generator=gen)) + 0.2).to(dt).cuda()[:, :H]
    res = r(R, H + 2 * pad).to(dt).cuda()[:, :H]
    w, b = (1 + 0.1 * r(H)).to(dt).cuda(), (0.1 * r(H)).to(dt).cuda()
    return x, res, w, b, r(R, H).to(dt).cuda(), r(R, H).to(dt).cuda()


CASES = [  # rows, columns: one value a lane to several vectors a thread, odd row counts
    (1, 8), (3, 16), (7, 64), (130, 96), (33, 256), (65, 264), (1, 4096), (1000, 520), (9, 2304), (5, 5000),
    (700, 1024), (3, 8192), (2, 16384), (4, 16376), (2500, 128),
    (20003, 1032),  # many rows for each block that is there at once
]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,H", CASES)
def test_forward_and_backward(R, H, dtype, rms, residual):
    from linear_cross_entropy_logit_gb300 import binding as B
    x, res, w, b, dy, ds = make(R, H, dtype, seed=R + H, pad=8)
    if not residual:
        res = ds = None
    y, s, mean, rstd = B.flce_layer_norm_forward(x, w, b, EPS, residual=res, rms=rms)
    if residual:
        want = tensor_f64(x) + tensor_f64(res)
        # one rounding to the type, of a sum rounded to fp32
        assert (np.abs(tensor_f64(s) - want) <= (2.0**-8 * 1.001 if dtype == "bf16" else 2.0**-24) * np.abs(want)).all()
    else:
        assert s is x
    wy, wm, wr = S.layer_norm_forward(tensor_f64(s), tensor_f64(w), tensor_f64(b), EPS, rms)
    assert near(y, wy, dtype) and rel_fro(tensor_f64(rstd), wr) <= TOL
    assert mean is None if rms else np.abs(tensor_f64(mean) - wm).max() <= TOL * np.abs(tensor_f64(s)).max()
    import torch
    nan = lambda *shape: torch.full(shape, float("nan"), device="cuda")  # noqa: E731
    ws = torch.full((2 * 152 * 32 * max(H, 128) * 4 + (1 << 22),), 255, dtype=torch.uint8, device="cuda")
    dx, dw, db = B.flce_layer_norm_backward(dy, s, w, mean, rstd, dsum=ds, rms=rms, dx=nan(R, H).to(dy.dtype),
                                            dweight=nan(H), dbias=nan(H), workspace_buf=ws)
    wx, ww, wb = S.layer_norm_backward(tensor_f64(dy), tensor_f64(s), tensor_f64(w), EPS,
                                       None if ds is None else tensor_f64(ds), rms)
    if H > 8:
        assert near(dx, wx, dtype)
    else:  # eight values: dx is a difference of terms up to rstd |dy| in size
        size = (rstd[:, None].abs() * dy.float().abs().amax(-1, keepdim=True) * 4).cpu().double().numpy()
        assert (np.abs(tensor_f64(dx) - wx) <= TOL * size + (2.0**-8 * np.abs(wx) if dtype == "bf16" else 0)).all()
    assert rel_fro(tensor_f64(dw), ww) <= TOL and rel_fro(tensor_f64(db), wb) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_without_weight_and_bias(dtype):
    from linear_cross_entropy_logit_gb300 import binding as B
    x, _, w, b, dy, _ = make(20, 72, dtype, seed=5)
    for weight, bias in ((None, None), (w, None), (None, b)):
        y, _, mean, rstd = B.flce_layer_norm_forward(x, weight, bias, EPS)
        f = lambda t: None if t is None else tensor_f64(t)  # noqa: E731
        assert near(y, S.layer_norm_forward(f(x), f(weight), f(bias), EPS)[0], dtype)
        dx, dw, db = B.flce_layer_norm_backward(dy, x, weight, mean, rstd, bias=bias is not None)
        wx, ww, wb = S.layer_norm_backward(f(dy), f(x), f(weight), EPS)
        assert near(dx, wx, dtype) and rel_fro(f(dw), ww) <= TOL
        assert db is None if bias is None else rel_fro(f(db), wb) <= TOL


def test_a_large_mean_does_not_swallow_the_spread():
    """The variance is summed from differences to the mean.  With a mean of 1000 spreads the
    inputs themselves are exact; the mean is off by up to 42 * 2^-24 of itself, 2.5e-3
    spreads, were its sum not a tree; over 2048 values its roundings add up in square: 7 *
    2^-24 * 1000 = 4e-4 spreads at most."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    gen = torch.Generator().manual_seed(7)
    x = (1000 + torch.randn(6, 2048, generator=gen)).cuda()
    y, _, mean, rstd = B.flce_layer_norm_forward(x, None)
    want, _, wr = S.layer_norm_forward(tensor_f64(x), None, None, 1e-5)
    assert np.abs(tensor_f64(y) - want).max() <= 4e-4 * 1.1 and rel_fro(tensor_f64(rstd), wr) <= 1e-5


def test_rows_do_not_touch_each_other():
    """NaN and infinities stay in their rows; a row of zeros norms to the bias."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    x, res, w, b, dy, ds = make(40, 264, "bf16", seed=8)
    x, bad = x.clone(), x.clone()
    bad[3, 5], bad[17, 0], bad[39, 263] = float("nan"), float("inf"), -float("inf")
    bad[20] = 0
    out = [B.flce_layer_norm_forward(t, w, b, EPS) for t in (x, bad)]
    keep = [i for i in range(40) if i not in (3, 17, 39, 20)]
    for a, c in ((out[0][0], out[1][0]), (out[0][2], out[1][2]), (out[0][3], out[1][3])):
        assert torch.equal(a[keep], c[keep])
    assert torch.equal(out[1][0][20], b) and out[1][0][[3, 17, 39]].isnan().any(-1).all()
    g = [B.flce_layer_norm_backward(dy, t, w, o[2], o[3], dsum=ds)[0] for t, o in zip((x, bad), out)]
    assert torch.equal(g[0][keep], g[1][keep]) and g[1][20].isfinite().all()


def test_in_place_and_given_outputs():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    for dtype in ("bf16", "fp32"):
        x, res, w, b, dy, ds = make(50, 512, dtype, seed=9)
        y, s, mean, rstd = B.flce_layer_norm_forward(x, w, b, EPS, residual=res)
        acc = res.clone()
        y2, s2, _, _ = B.flce_layer_norm_forward(x, w, b, EPS, residual=acc, sum_out=acc)
        assert s2 is acc and torch.equal(acc, s) and torch.equal(y2, y)
        dx, dw, db = B.flce_layer_norm_backward(dy, s, w, mean, rstd, dsum=ds)
        g = ds.clone()
        dx2, dw2, _ = B.flce_layer_norm_backward(dy, s, w, mean, rstd, dsum=g, dx=g)
        assert dx2 is g and torch.equal(g, dx) and torch.equal(dw, dw2)
        g = dy.clone()
        B.flce_layer_norm_backward(g, s, w, mean, rstd, dsum=ds, dx=g)
        assert torch.equal(g, dx)
        acc = x.contiguous().clone()
        B.flce_layer_norm_forward(acc, w, b, EPS, residual=res, sum_out=acc)
        assert torch.equal(acc, s)


def test_no_rows_and_same_bits():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    x, res, w, b, dy, ds = make(0, 64, "fp32")
    y, s, mean, rstd = B.flce_layer_norm_forward(x, w, b, EPS, residual=res)
    dx, dw, db = B.flce_layer_norm_backward(dy, s, w, mean, rstd, dweight=torch.ones(64, device="cuda"))
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()
    x, res, w, b, dy, ds = make(3001, 1032, "bf16", seed=11)
    _, s, mean, rstd = B.flce_layer_norm_forward(x, w, b, EPS)
    first, *others = [B.flce_layer_norm_backward(dy, s, w, mean, rstd) for _ in range(3)]
    assert all(torch.equal(p, q) for o in others for p, q in zip(first, o))


def test_autograd_sum_used_or_not():
    """Gradients through y, through the sum, and through either alone; shapes with leading
    dimensions; on another stream."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    gen = torch.Generator().manual_seed(12)
    x, r = (torch.randn(4, 9, 40, generator=gen, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(40, generator=gen, dtype=torch.float64) for _ in range(2))
    side = torch.cuda.Stream()
    for use_y, use_s in ((1, 1), (1, 0), (0, 1)):
        p = [t.clone().requires_grad_() for t in (x, r, w, b)]
        s = p[0] + p[1]
        y = torch.nn.functional.layer_norm(s, (40,), p[2], p[3], 1e-5)
        (use_y * y.pow(2).sum() + use_s * s.pow(3).sum()).backward()
        with torch.cuda.stream(side):
            q = [t.float().cuda().requires_grad_() for t in (x, r, w, b)]
            y, s = B.layer_norm(q[0], q[2], q[3], residual=q[1])
            total = 0
            if use_y:
                total = total + y.pow(2).sum()
            if use_s:
                total = total + s.pow(3).sum()
            total.backward()
        side.synchronize()
        for a, c in zip(q, p):
            if a.grad is None:
                assert not use_y and c.grad.abs().max() == 0
            else:
                assert rel_fro(tensor_f64(a.grad), c.grad.numpy()) <= 2e-5
    y = B.layer_norm(q[0].detach(), q[2].detach(), rms=True)
    assert y.shape == x.shape
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g,) = torch.autograd.grad(B.layer_norm(q[0], q[2]).pow(2).sum(), q[0], create_graph=True)
        g.sum().backward()


def test_replay_in_a_graph():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    x, res, w, b, dy, ds = make(300, 2304, "bf16", seed=13)
    x, res = x.clone(), res.clone()

    def step():
        y, s, mean, rstd = B.flce_layer_norm_forward(x, w, b, EPS, residual=res)
        return y, s, *B.flce_layer_norm_backward(dy, s, w, mean, rstd, dsum=ds)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for scale in (2.0, -0.5):
        x.mul_(scale)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))
