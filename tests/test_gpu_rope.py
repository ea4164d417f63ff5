"""Rotary positions against the fp64 oracle.

Tolerances: cosine and sine of an angle rounded to 2^-25 of half a turn (1e-7), their own
last bits (2 * 2^-24), two products and a sum: below 4e-7 of a pair's length, 1e-6 in all.
A bf16 output adds one rounding, 2^-8 of its value."""
import math

import numpy as np
import pytest

from oracle import step_oracle as S
from tests.gpu_util import tensor_f64

pytestmark = pytest.mark.gpu


def near(got, want, x, dtype, magnitude=1.0):
    err = np.abs(tensor_f64(got) - want)
    if dtype == "bf16":
        err = np.maximum(0.0, err - 2.0**-8 * np.abs(want))
    return (err <= 1e-6 * magnitude * math.sqrt(2.0) * np.abs(x).max()).all()


def make(T, HQ, HK, D, dtype, seed=0, fused=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    qkv = torch.randn(T, HQ + 2 * HK, D + (8 if fused else 0), generator=gen).to(dt).cuda()
    q, k = qkv[:, :HQ, :D], qkv[:, HQ:HQ + HK, :D]
    return (q, k) if fused else (q.contiguous(), k.contiguous())


CASES = [  # T, HQ, HK, D, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 8, 8), (37, 3, 1, 64, 64), (130, 14, 2, 80, 40), (65, 5, 5, 96, 96),
    (33, 4, 2, 128, 32), (19, 2, 1, 256, 128), (12, 6, 2, 136, 136), (50, 4, 4, 72, 24), (3000, 7, 1, 128, 128),
    (5, 90, 40, 256, 256), (2, 300, 3, 16, 16),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,HQ,HK,D,rot", CASES)
def test_forward_and_backward(T, HQ, HK, D, rot, dtype, interleaved):
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(T, HQ, HK, D, dtype, seed=T + D)
    inv, m = B.rope_frequencies(rot, 10000.0, "yarn", factor=4.0, trained_length=2048)
    pos = torch.randint(-5, 200000, (T,), generator=torch.Generator().manual_seed(1)).cuda()
    f = inv.cpu().numpy()
    for back, call in ((False, B.flce_rope_forward), (True, B.flce_rope_backward)):
        out = call(q, k, inv, pos, magnitude=m, interleaved=interleaved)
        for got, x in zip(out, (q, k)):
            want = S.rope(tensor_f64(x), f, pos.tolist(), np.float32(m), interleaved, back)
            assert got.is_contiguous() and near(got, want, tensor_f64(x), dtype, m)
            assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("start", [0, 10**6, 2**31 - 3, 2**40, -(2**33)])
def test_far_positions_are_as_exact(start):
    """The frequencies are multiples of 2^-20 turns: their angles are known exactly at any
    position."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(6, 2, 1, 64, "fp32", seed=4, fused=False)
    pos = torch.arange(6) + start
    parts = [(2 * j + 1) * 97 % 2**20 for j in range(32)]  # of 2^20 a turn
    inv = torch.tensor([p / 2**20 * 2 * math.pi for p in parts], dtype=torch.float64).cuda()
    qo, _ = B.flce_rope_forward(q, k, inv, pos.cuda())
    turns = np.array([[(int(p) * n % 2**20) / 2**20 for n in parts] for p in pos.tolist()])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    x = tensor_f64(q)
    a, b = x[..., :32], x[..., 32:]
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    # inv / 2 pi is off by 2^-52 of itself at most, twice rounded: so many turns at this position
    drift = 2 * np.pi * abs(start + 6) * 2.0**-52 * max(parts) / 2**20
    assert np.abs(tensor_f64(qo) - want).max() <= (1e-6 + drift) * math.sqrt(2.0) * np.abs(x).max()


def test_default_positions_in_place_and_autograd():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(70, 4, 2, 64, "fp32", seed=3, fused=False)
    inv, _ = B.rope_frequencies(32)
    want = B.flce_rope_forward(q, k, inv, torch.arange(70, device="cuda"), interleaved=True)
    got = B.flce_rope_forward(q, k, inv, interleaved=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b = q.clone(), k.clone()
    B.flce_rope_forward(a, b, inv, interleaved=True, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    # gradients, one of them broadcast, from another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lq, lk = q.clone().requires_grad_(), k.clone().requires_grad_()
        oq, ok = B.rope(lq, lk, inv, magnitude=1.5)
        gq = torch.randn_like(oq)
        torch.autograd.backward((oq, ok), (gq, torch.ones(1, 1, 1, device="cuda").expand_as(ok)))
    side.synchronize()
    f, pos = inv.cpu().numpy(), range(70)
    assert near(lq.grad, S.rope(tensor_f64(gq), f, pos, 1.5, False, True), tensor_f64(gq), "fp32", 1.5)
    ones = np.ones(k.shape)
    assert near(lk.grad, S.rope(ones, f, pos, 1.5, False, True), ones, "fp32", 1.5)


def test_no_tokens():
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(0, 4, 2, 64, "bf16")
    inv, _ = B.rope_frequencies(64)
    qo, ko = B.flce_rope_forward(q, k, inv)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)


def test_what_is_not_finite_stays_in_its_pair():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(5, 2, 1, 64, "bf16", seed=6, fused=False)
    inv, _ = B.rope_frequencies(48)
    want, _ = B.flce_rope_forward(q, k, inv)
    bad = q.clone()
    bad[2, 1, 3], bad[4, 0, 50] = float("nan"), float("inf")
    got, _ = B.flce_rope_forward(bad, k, inv)
    same = torch.ones_like(q, dtype=torch.bool)
    same[2, 1, 3] = same[2, 1, 27] = same[4, 0, 50] = False
    assert torch.equal(got[same], want[same]) and got[4, 0, 50] == float("inf") and got[2, 1, 27].isnan()


def test_any_frequency():
    """Negative and large ones turn as the formula says, zero not at all; one that is not
    finite makes its pairs NaN and no others."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k = make(7, 2, 1, 16, "fp32", seed=7, fused=False)
    pos = torch.tensor([0, 1, -3, 50, 999, 12345, -7], device="cuda")
    f = [-0.25, 30.0, 0.0, 6.5, 1e-9, -12.0, 2.0**-70, 1.0]
    qo, _ = B.flce_rope_forward(q, k, torch.tensor(f, dtype=torch.float64, device="cuda"), pos)
    assert near(qo, S.rope(tensor_f64(q), f, pos.tolist()), tensor_f64(q), "fp32")
    for bad in (float("nan"), float("inf")):
        f[3] = bad
        got, _ = B.flce_rope_forward(q, k, torch.tensor(f, dtype=torch.float64, device="cuda"), pos)
        same = [i for i in range(16) if i % 8 != 3]
        assert got[..., [3, 11]].isnan().all() and torch.equal(got[..., same], qo[..., same])
