"""The attention block under the fused loss (examples/packed_training_step.py) against
the same step in plain fp64 torch operations, and the example's command."""
import math
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain_step(block, x, cu, positions, labels):
    """loss and gradients in fp64, every operation spelled out."""
    import torch
    P = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    q_heads, kv_heads, dim = block.shape
    T = x.shape[0]
    x = x.double()
    q, k, v = (x @ P["qkv"].T).view(T, -1, dim).split([q_heads, kv_heads, kv_heads], 1)
    cos, sin = (t.double()[positions][:, None] for t in (block.cos, block.sin))

    def normed(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = t.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = normed(q, P["q_norm"]), normed(k, P["k_norm"])
    group = q_heads // kv_heads
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    of = torch.bucketize(torch.arange(T, device=x.device), cu[1:].long(), right=True)
    seen = (of[:, None] == of) & (torch.arange(T, device=x.device)[:, None] >= torch.arange(T, device=x.device))
    s = torch.einsum("thd,uhd->htu", q, k) / math.sqrt(dim)
    p = s.masked_fill(~seen, -math.inf).softmax(-1)
    a = torch.einsum("htu,uhd->thd", p, v)
    h = x + a.reshape(T, -1) @ P["out"].T
    logits = h @ P["vocab"].T
    loss = torch.nn.functional.cross_entropy(logits, labels, ignore_index=-100)
    loss.backward()
    return loss.item(), {n: p.grad for n, p in P.items()}


def test_block_matches_plain_fp64():
    import torch
    from packed_training_step import Block, packed_batch
    torch.manual_seed(1)
    block = Block(256, 8, 2, 64, 1000, 400)
    with torch.no_grad():
        block.q_norm += 0.1 * torch.randn_like(block.q_norm)
    x, cu, positions, labels = packed_batch(397, 5, 256, 1000)
    loss = block(x, cu, positions, labels)
    loss.backward()
    want, grads = plain_step(block, x, cu, positions, labels)
    # the loss's own bar; gradients pass through up to eight roundings to bf16 (projections, heads,
    # attention, hidden states and their gradients) of 2^-9 / sqrt(3) on average each, which add up
    # in square: sqrt(8) * 1.1e-3 = 3e-3 of the unrounded size, and the gradients of q and k are small
    # differences of larger terms, which an order of magnitude covers
    assert abs(loss.item() - want) <= 2e-3 * abs(want)
    for name, p in block.named_parameters():
        g = grads[name]
        assert (p.grad.double() - g).norm() <= 3e-2 * g.norm(), name


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "packed_training_step.py"),
                        "--tokens", "600", "--sequences", "3", "--hidden", "256", "--q-heads", "4",
                        "--kv-heads", "2", "--head-dim", "64", "--vocab", "2000", "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split("loss ")[1].split(",")[0]) for line in r.stdout.splitlines()]
    assert len(losses) == 3 and losses[-1] < losses[0]


@pytest.mark.parametrize("T,HQ,HK,D,cuts", [(40, 4, 2, 64, [0, 13, 40]), (700, 6, 2, 128, [0, 5, 300, 690]),
                                            (2600, 8, 2, 64, [0, 2600])])
def test_calls_in_a_row_see_each_others_results(T, HQ, HK, D, cuts):
    """Each launch may start while the one before it ends: a chain of calls that read
    what the last ones wrote, into the same buffers, gives the bits of calls made one by one."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    gen = torch.Generator().manual_seed(T)

    def r(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen).to("cuda", dtype)

    x = [r(T, HQ, D), r(T, HK, D)]
    w = [r(D), r(D)]
    angle = r(T, D // 2, dtype=torch.float32)
    cos, sin = angle.cos(), angle.sin()
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")

    def chain(wait):
        q, k = x[0].clone(), x[1].clone()
        v = x[1].flip(0).contiguous()
        a, b, out, dq, dk, dv = (torch.empty_like(t) for t in (q, k, q, q, k, k))
        lse = torch.empty(HQ, T, device="cuda")
        dw = [torch.empty(D, device="cuda") for _ in range(2)]
        err = B.new_err_word("cuda")
        kept = []
        wait()
        for i in range(12):
            B.flce_qk_norm_rope_forward(q, k, *w, cos, sin, q_out=a, k_out=b, err_word=err)
            wait()
            B.flce_attention_forward(a, b, v, cu, out=out, lse=lse, err_word=err)
            wait()
            B.flce_attention_backward(a, a, b, v, out, lse, cu, dq=dq, dk=dk, dv=dv, err_word=err)
            wait()
            # the next step's inputs: q and k from their gradients
            B.flce_qk_norm_rope_backward(dq, dk, a, b, *w, cos, sin, dq=q, dk=k, dq_weight=dw[0],
                                         dk_weight=dw[1], err_word=err)
            wait()
            if i % 4 == 3:
                kept += [t.clone() for t in (q, k, out, lse, dv, *dw)]
                wait()
        assert int(err.item()) == 0
        return kept

    want = chain(torch.cuda.synchronize)
    for _ in range(4):
        got = chain(lambda: None)
        assert all(torch.equal(p.nan_to_num(), t.nan_to_num()) for p, t in zip(got, want))
    assert all(t[..., :cuts[-1], :].isfinite().all() for t in want if t.dim() == 3)


def test_second_derivatives_are_refused():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q, k, v = (torch.randn(9, 2, 64, device="cuda").bfloat16().requires_grad_() for _ in range(3))
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    out = B.packed_attention(*B.qk_norm_rope(q, k, None, None, None, None), v, cu)
    (g,) = torch.autograd.grad(out.float().pow(2).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()
