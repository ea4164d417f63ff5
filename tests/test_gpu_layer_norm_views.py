"""Weights of a layer norm that start anywhere (views of one flat buffer of parameters)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rms", [False, True])
def test_weights_off_their_alignment(rms, dtype):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    flat = torch.randn(1 + 2 * 130, device="cuda").to(dt).requires_grad_()
    x = torch.randn(10, 128, device="cuda").to(dt)
    results = []
    for views in (True, False):
        w, b = flat[1:129], flat[131:259]
        if not views:
            w, b = w.detach().clone().requires_grad_(), b.detach().clone().requires_grad_()
        y, s = B.layer_norm(x, w, b, residual=x, rms=rms)
        gw, gb = torch.autograd.grad(y.float().pow(2).sum() + s.float().sum(), (w, b))
        results.append((y, s, gw, gb))
    for a, c in zip(*results):
        assert torch.equal(a, c)
    # every other value of a buffer
    y, _ = B.layer_norm(x, flat[::2][:128], None, residual=x, rms=rms)
    want, _ = B.layer_norm(x, flat[::2][:128].contiguous(), None, residual=x, rms=rms)
    assert torch.equal(y, want)
    assert torch.autograd.grad(y.float().sum(), flat)[0][1::2].abs().max() == 0
