"""One training step of a pre-norm attention block under a teacher's top logits, on a packed batch.

    python examples/distillation_step.py [--tokens 8192] [--sequences 4] ...

Hidden states of several packed sequences go through one block without head norms (RMS norm,
projection, rotary positions scaled past the trained length, causal attention within each
sequence, output projection, the residual sum with the norm behind it) and the linear
distillation from the top logits of a teacher; the gradients of every weight come back.  The
projections are plain matrix products; everything between and after them is the library's.
Tokens of the prompts have no entries.  Synthetic data.
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
    """A pre-norm attention block and the unembedding matrix behind it."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, vocab, theta=500000.0, factor=8.0,
                 trained_length=8192, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.shape = (q_heads, kv_heads, head_dim)

        def weight(*size):
            return torch.nn.Parameter(0.02 * torch.randn(*size, device=device, dtype=dtype))

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        self.vocab = weight(vocab, hidden)
        self.norm_in = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.norm_out = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        inv_freq, self.magnitude = B.rope_frequencies(head_dim, theta, "llama3", factor=factor,
                                                      trained_length=trained_length, device=device)
        self.register_buffer("inv_freq", inv_freq)

    def forward(self, x, cu_seqlens, positions, err_word=None):
        """The hidden states in front of the unembedding."""
        q_heads, kv_heads, dim = self.shape
        h = B.layer_norm(x, self.norm_in, rms=True)
        # q, k and v are views of the projection's output
        q, k, v = (h @ self.qkv.T).view(x.shape[0], -1, dim).split([q_heads, kv_heads, kv_heads], 1)
        q, k = B.rope(q, k, self.inv_freq, positions, magnitude=self.magnitude)
        a = B.packed_attention(q, k, v, cu_seqlens, err_word=err_word)
        y, _ = B.layer_norm(a.reshape(x.shape[0], -1) @ self.out.T, self.norm_out, residual=x, rms=True)
        return y


@torch.no_grad()
def top_logits(teacher, batch, top, rows=1024):
    """ids and logits of the teacher's `top` largest logits of each token, some tokens at a time."""
    h = teacher(*batch)
    parts = [(h[i:i + rows] @ teacher.vocab.T).float().topk(top) for i in range(0, h.shape[0], rows)]
    return torch.cat([p.indices for p in parts]), torch.cat([p.values for p in parts])


def packed_batch(tokens, sequences, hidden, seed=0, dtype=torch.bfloat16, device="cuda"):
    """(hidden states, offsets, positions within the sequences), and which tokens are a prompt's."""
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.randperm(tokens - 1, generator=gen)[: sequences - 1].sort().values + 1
    cu = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([tokens])])
    positions = torch.arange(tokens) - cu[:-1].repeat_interleave(cu.diff())
    prompt = positions < (cu.diff() // 4).repeat_interleave(cu.diff())
    x = torch.randn(tokens, hidden, generator=gen)
    return (x.to(device, dtype), cu.to(device, torch.int32), positions.to(device)), prompt.to(device)


def step(block, batch, ids, logits, temperature, err_word=None):
    """The loss, and its gradients in the block's parameters."""
    loss = B.linear_distillation(block(*batch, err_word), block.vocab, ids, logits, temperature, err_word=err_word)
    loss.backward()
    return loss


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 8192), ("sequences", 4), ("hidden", 4096), ("q-heads", 32),
                          ("kv-heads", 8), ("head-dim", 128), ("vocab", 128256), ("top", 64), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args()
    torch.manual_seed(0)
    shape = (a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.vocab)
    teacher, block = Block(*shape), Block(*shape)
    opt = torch.optim.SGD(block.parameters(), lr=0.1)
    batch, prompt = packed_batch(a.tokens, a.sequences, a.hidden)
    ids, logits = top_logits(teacher, batch, a.top)
    ids[prompt] = -1
    err = B.new_err_word("cuda")
    for n in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        opt.zero_grad(set_to_none=True)
        loss = step(block, batch, ids, logits, a.temperature, err)
        opt.step()
        torch.cuda.synchronize()
        if err.item():
            raise B.FlceError(err.item(), "distillation step")
        print(f"step {n}: loss {loss.item():.4f}, {1e3 * (time.perf_counter() - t):.2f} ms", flush=True)


if __name__ == "__main__":
    main()
