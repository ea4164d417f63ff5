"""One training step of an attention block under the fused loss, on a packed batch.

    python examples/packed_training_step.py [--tokens 8192] [--sequences 4] ...

Hidden states of several packed sequences go through one attention block
(projection, per-head norm with rotary positions, causal attention within each
sequence, output projection, residual) and the fused linear cross-entropy; the
gradients of every weight come back.  The projections are plain matrix
products; everything between and after them is the library's.  Tokens of the
prompts are ignored by the loss (label -100).  Synthetic data.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from linear_cross_entropy_logit_gb300 import binding as B  # noqa: E402


class Block(torch.nn.Module):
    """An attention block and the unembedding matrix of the loss behind it."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, vocab, positions, theta=10000.0,
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.shape = (q_heads, kv_heads, head_dim)

        def weight(*size):
            return torch.nn.Parameter(0.02 * torch.randn(*size, device=device, dtype=dtype))

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        self.vocab = weight(vocab, hidden)
        self.q_norm = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))
        self.k_norm = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))
        freq = theta ** (-torch.arange(0, head_dim, 2, device=device, dtype=torch.float64) / head_dim)
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
        self.register_buffer("cos", angle.cos().float())
        self.register_buffer("sin", angle.sin().float())

    def forward(self, x, cu_seqlens, positions, labels, err_word=None):
        q_heads, kv_heads, dim = self.shape
        # q, k and v are views of the projection's output
        q, k, v = (x @ self.qkv.T).view(x.shape[0], -1, dim).split([q_heads, kv_heads, kv_heads], 1)
        q, k = B.qk_norm_rope(q, k, self.q_norm, self.k_norm, self.cos, self.sin, positions,
                              err_word=err_word)
        a = B.packed_attention(q, k, v, cu_seqlens, err_word=err_word)
        h = x + a.reshape(x.shape[0], -1) @ self.out.T
        return B.linear_cross_entropy(h, self.vocab, labels, ignore_index=-100)


def packed_batch(tokens, sequences, hidden, vocab, seed=0, dtype=torch.bfloat16, device="cuda"):
    """Hidden states, offsets, positions within the sequences, and labels with ignored prompts."""
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.randperm(tokens - 1, generator=gen)[: sequences - 1].sort().values + 1
    cu = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([tokens])])
    starts = cu[:-1].repeat_interleave(cu.diff())
    positions = torch.arange(tokens) - starts
    labels = torch.randint(vocab, (tokens,), generator=gen)
    labels[positions < (cu.diff() // 4).repeat_interleave(cu.diff())] = -100
    x = torch.randn(tokens, hidden, generator=gen)
    return (x.to(device, dtype), cu.to(device, torch.int32), positions.to(device), labels.to(device))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 8192), ("sequences", 4), ("hidden", 4096), ("q-heads", 32),
                          ("kv-heads", 8), ("head-dim", 128), ("vocab", 128256), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    torch.manual_seed(0)
    block = Block(a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.vocab, a.tokens)
    opt = torch.optim.SGD(block.parameters(), lr=0.1)
    batch = packed_batch(a.tokens, a.sequences, a.hidden, a.vocab)
    err = B.new_err_word("cuda")
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        opt.zero_grad(set_to_none=True)
        loss = block(*batch, err)
        loss.backward()
        opt.step()
        torch.cuda.synchronize()
        if err.item():
            raise B.FlceError(err.item(), "packed training step")
        print(f"step {step}: loss {loss.item():.4f}, {1e3 * (time.perf_counter() - t):.2f} ms", flush=True)


if __name__ == "__main__":
    main()
