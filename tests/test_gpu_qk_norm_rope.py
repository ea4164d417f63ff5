"""Head norm with rotary positions against the fp64 oracle.

Tolerances: all arithmetic is fp32 with about 30 roundings from input to
output, so fp32 results are within a few 2^-23 of the oracle (1e-5 leaves room
for sums over thousands of heads in the weights' gradients); a bf16 output adds
one rounding to nearest, at most 2^-8 of its own value."""
import numpy as np
import pytest

from oracle import attn_oracle as A
from tests.gpu_util import rel_fro, tensor_f64

pytestmark = pytest.mark.gpu
TOL = 1e-5
EPS = 1e-6


def near(got, want, dtype):
    """fp32 within TOL in relative Frobenius norm; bf16 within one rounding of each value
    on top of that."""
    err = np.abs(tensor_f64(got) - want)
    if dtype == "bf16":
        err = np.maximum(0.0, err - 2.0**-8 * np.abs(want))
    return np.linalg.norm(err) <= TOL * np.linalg.norm(want)


def make(T, HQ, HK, D, rot, dtype, seed=0, rows=64, fused=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    pad = 8 if fused else 0
    qkv = r(T, HQ + 2 * HK, D + pad).to(dt).cuda()
    q, k = qkv[:, :HQ, :D], qkv[:, HQ:HQ + HK, :D]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.1 * r(D)).to(dt).cuda() for _ in range(2)]
    angle = 6.0 * torch.rand(rows, rot // 2, generator=gen)
    tables = [angle.cos().cuda(), angle.sin().cuda()] if rot else [None, None]
    pos = torch.randint(0, rows, (T,), generator=gen).cuda()
    grads = [r(T, h, D).to(dt).cuda() for h in (HQ, HK)]
    return q, k, w, tables, pos, grads


def oracle(q, k, w, tables, pos, grads, rot, interleaved):
    T = q.shape[0]
    cos, sin = [tensor_f64(t) if t is not None else np.zeros((64, 0)) for t in tables]
    p = pos.cpu().numpy() if pos is not None else np.arange(T)
    out = []
    for x, wt, g in zip((q, k), w, grads):
        wt = tensor_f64(wt) if wt is not None else np.ones(x.shape[-1])
        a = (cos, sin, p, EPS, interleaved)
        dx, dw = A.qk_norm_rope_backward(tensor_f64(g), tensor_f64(x), wt, *a)
        out.append((A.qk_norm_rope_forward(tensor_f64(x), wt, *a), dx, dw))
    return out


CASES = [  # T, HQ, HK, D, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 8, 8), (37, 3, 1, 64, 64), (130, 14, 2, 80, 40),
    (65, 5, 5, 96, 96), (33, 4, 2, 128, 32), (19, 2, 1, 256, 128), (12, 6, 2, 136, 136),
    (50, 4, 4, 72, 0), (3000, 7, 1, 128, 128),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,HQ,HK,D,rot", CASES)
def test_forward_and_backward(T, HQ, HK, D, rot, dtype, interleaved):
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(T, HQ, HK, D, rot, dtype, seed=T)
    qo, ko, err = B.flce_qk_norm_rope_forward(q, k, *w, *tables, pos, EPS, interleaved=interleaved)
    dq, dk, dwq, dwk, _ = B.flce_qk_norm_rope_backward(*grads, q, k, *w, *tables, pos, EPS,
                                                       interleaved=interleaved, err_word=err)
    (yq, xq, gq), (yk, xk, gk) = oracle(q, k, w, tables, pos, grads, rot, interleaved)
    assert int(err.item()) == 0
    for got, want in ((qo, yq), (ko, yk), (dq, xq), (dk, xk)):
        assert near(got, want, dtype)
    for got, want in ((dwq, gq), (dwk, gk)):
        assert rel_fro(tensor_f64(got), want) <= 1e-5


def test_no_weights_default_positions_and_contiguous_inputs():
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, _, tables, _, grads = make(40, 4, 2, 64, 32, "fp32", seed=3, fused=False)
    qo, ko, err = B.flce_qk_norm_rope_forward(q, k, None, None, *tables)
    (yq, _, _), (yk, _, _) = oracle(q, k, [None, None], tables, None, grads, 32, False)
    assert int(err.item()) == 0
    assert rel_fro(tensor_f64(qo), yq) <= 1e-5 and rel_fro(tensor_f64(ko), yk) <= 1e-5


def test_position_outside_the_tables_is_reported_and_left_unrotated():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(9, 2, 1, 64, 64, "fp32", seed=4)
    pos[3], pos[7] = 64, -1
    qo, _, err = B.flce_qk_norm_rope_forward(q, k, *w, *tables, pos)
    still = [torch.ones_like(tables[0]), torch.zeros_like(tables[1])]  # an angle of zero
    plain, _, _ = B.flce_qk_norm_rope_forward(q, k, *w, *still)
    assert int(err.item()) == B.FLCE_ERR_INDEX
    assert (qo[[3, 7]] == plain[[3, 7]]).all() and not (qo[[2, 4]] == plain[[2, 4]]).all()


def test_no_tokens():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(0, 2, 1, 64, 64, "bf16")
    qo, ko, _ = B.flce_qk_norm_rope_forward(q, k, *w, *tables, pos)
    dwq, dwk = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    B.flce_qk_norm_rope_backward(*grads, q, k, *w, *tables, pos, dq_weight=dwq, dk_weight=dwk)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)
    assert not dwq.any() and not dwk.any()


def test_zero_rows_and_extremes_stay_finite():
    """A head of zeros norms to zeros (eps > 0); 1e4-sized heads do not overflow."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(5, 2, 1, 128, 128, "bf16", seed=6, fused=False)
    q[2] = 0
    q[3] *= 1e4
    qo, _, _ = B.flce_qk_norm_rope_forward(q, k, *w, *tables, pos)
    assert not qo[2].any() and torch.isfinite(qo).all()


def test_runs_give_the_same_bits():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(2000, 8, 2, 128, 128, "bf16", seed=8)
    r = [B.flce_qk_norm_rope_backward(*grads, q, k, *w, *tables, pos)[:4] for _ in range(3)]
    for other in r[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r[0], other))


def test_autograd_on_another_stream():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, w, tables, pos, grads = make(100, 4, 2, 64, 64, "fp32", seed=9)
    leaves = [t.clone().requires_grad_() for t in (q, k, *w)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qo, ko = B.qk_norm_rope(*leaves, *tables, pos)
        torch.autograd.backward((qo, ko), grads)
    torch.cuda.current_stream().wait_stream(s)
    (yq, xq, gq), (yk, xk, gk) = oracle(q, k, w, tables, pos, grads, 64, False)
    for got, want in ((qo, yq), (leaves[0].grad, xq), (leaves[1].grad, xk),
                      (leaves[2].grad, gq), (leaves[3].grad, gk)):
        assert rel_fro(tensor_f64(got), want) <= 1e-5
