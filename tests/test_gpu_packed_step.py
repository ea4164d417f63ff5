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
