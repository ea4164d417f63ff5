"""The block under a teacher's top logits (examples/distillation_step.py) against the same step
in plain fp64 torch operations, a chain of overlapping calls, and the example's command."""
import math
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain_step(block, x, cu, positions, ids, logits, temperature):
    """loss and gradients in fp64, every operation spelled out."""
    import torch
    P = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    q_heads, kv_heads, dim = block.shape
    T, x = x.shape[0], x.double()

    def normed(t, w):
        return t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w

    q, k, v = (normed(x, P["norm_in"]) @ P["qkv"].T).view(T, -1, dim).split([q_heads, kv_heads, kv_heads], 1)
    angle = positions.double()[:, None, None] * block.inv_freq

    def turned(t):
        a, b = t.chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    q, k = turned(q), turned(k)
    k, v = (t.repeat_interleave(q_heads // kv_heads, 1) for t in (k, v))
    at = torch.arange(T, device=x.device)
    of = torch.bucketize(at, cu[1:].long(), right=True)
    s = torch.einsum("thd,uhd->htu", q, k) / math.sqrt(dim)
    p = s.masked_fill((of[:, None] != of) | (at[:, None] < at), -math.inf).softmax(-1)
    a = torch.einsum("htu,uhd->thd", p, v).reshape(T, -1)
    h = normed(x + a @ P["out"].T, P["norm_out"])
    logp = (h @ P["vocab"].T / temperature).log_softmax(-1)
    there = ids >= 0
    logq = (logits.double() / temperature).masked_fill(~there, -math.inf)
    logq = (logq - logq.logsumexp(-1, keepdim=True))[there.any(-1)]
    rows = logq.exp() * (logq - logp.gather(1, ids.clamp(min=0))[there.any(-1)])
    loss = rows.sum() / there.any(-1).sum()
    loss.backward()
    return loss.item(), {n: p.grad for n, p in P.items()}


def test_block_matches_plain_fp64():
    import torch
    from distillation_step import Block, packed_batch, step, top_logits
    from linear_cross_entropy_logit_gb300 import binding as B
    torch.manual_seed(1)
    teacher, block = Block(256, 8, 2, 64, 1000), Block(256, 8, 2, 64, 1000)
    with torch.no_grad():
        for w in (block.norm_in, block.norm_out):
            w += 0.1 * torch.randn_like(w)
    batch, prompt = packed_batch(397, 5, 256)
    ids, logits = top_logits(teacher, batch, 20)
    ids[prompt] = -1
    err = B.new_err_word("cuda")
    loss = step(block, batch, ids, logits, 1.5, err)
    want, grads = plain_step(block, *batch, ids, logits, 1.5)
    # the hidden states in front of the loss are rounded to bf16 about five times on their way
    # (2^-9 / sqrt(3) each, 2.5e-3 together), the logits of size 1 with them: far below 2e-3 of a loss of
    # 5 after the mean over 300 tokens; gradients pass through up to ten such roundings, sqrt(10) *
    # 1.1e-3 = 3.6e-3 of the unrounded size, and those of q and k are small differences of larger
    # terms, which an order of magnitude covers
    assert int(err.item()) == 0 and abs(loss.item() - want) <= 2e-3 * abs(want)
    for name, p in block.named_parameters():
        g = grads[name]
        assert (p.grad.double() - g).norm() <= 3e-2 * g.norm(), name


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "distillation_step.py"),
                        "--tokens", "600", "--sequences", "3", "--hidden", "256", "--q-heads", "4",
                        "--kv-heads", "2", "--head-dim", "64", "--vocab", "2000", "--top", "9", "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split("loss ")[1].split(",")[0]) for line in r.stdout.splitlines()]
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)


@pytest.mark.parametrize("T,H,V,K,heads,D", [(40, 128, 600, 5, 2, 64), (700, 512, 3001, 33, 8, 64),
                                             (2600, 256, 9000, 16, 2, 128)])
def test_calls_in_a_row_see_each_others_results(T, H, V, K, heads, D):
    """Launches overlap the end of the ones before them: a chain of calls that read what the
    last ones wrote, into the same buffers, gives the bits of calls made one by one."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    assert heads * D <= H
    gen = torch.Generator().manual_seed(T)

    def r(*shape, dtype=torch.bfloat16, scale=1.0):
        return (scale * torch.randn(*shape, generator=gen)).to("cuda", dtype)

    x0, W, w = r(T, H), r(V, H, scale=0.05), r(H, scale=0.1) + 1
    ids = torch.randint(0, V, (T, K), generator=gen).cuda()
    t = r(T, K, dtype=torch.float32, scale=2.0)
    inv, _ = B.rope_frequencies(D)
    ws = torch.empty(B.flce_distill_workspace_size(T, H, V, K), dtype=torch.uint8, device="cuda")

    def chain(wait):
        x, y, s, dX, dx = x0.clone(), *(torch.empty_like(x0) for _ in range(4))
        mean, rstd, lse = (torch.empty(T, device="cuda") for _ in range(3))
        logits, dW = torch.empty(T, K, device="cuda"), torch.empty_like(W)
        dw, db, loss = torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(1, device="cuda")
        valid = torch.empty(1, dtype=torch.int32, device="cuda")
        err, kept = B.new_err_word("cuda"), []
        wait()
        for i in range(8):
            B.flce_layer_norm_forward(x, w, None, residual=x0, out=y, sum_out=s, mean=mean, rstd=rstd)
            wait()
            q = y[:, :heads * D].unflatten(1, (heads, D))
            q2, k2 = B.flce_rope_forward(q, q, inv)
            wait()
            y[:, :heads * D] = q2.flatten(1) + k2.flatten(1)
            wait()
            B.flce_distill_forward(y, W, ids, t, 1.3, loss=loss, lse=lse, logits=logits, valid_count=valid,
                                   workspace_buf=ws, err_word=err)
            wait()
            B.flce_distill_backward(y, W, ids, t, lse, logits, valid, 1.3, dX=dX, dW=dW, workspace_buf=ws,
                                    err_word=err)
            wait()
            B.flce_layer_norm_backward(dX, s, w, mean, rstd, dsum=y, dx=dx, dweight=dw, dbias=db)
            wait()
            x.copy_(dx)  # the next step's input
            wait()
            if i % 4 == 3:
                kept += [v.clone() for v in (x, loss, lse, logits, dW, dw, db)]
                wait()
        assert int(err.item()) == 0
        return kept

    want = chain(torch.cuda.synchronize)
    assert all(v.isfinite().all() for v in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))


def test_a_captured_step_replays():
    """Forward and gradients through autograd in a CUDA graph, on new inputs in the captured
    buffers: the bits of the same step made eagerly."""
    import torch
    from distillation_step import Block, packed_batch
    from linear_cross_entropy_logit_gb300 import binding as B
    torch.manual_seed(2)
    block = Block(256, 4, 2, 64, 1500)
    batch, prompt = packed_batch(300, 3, 256)
    ids = torch.randint(0, 1500, (300, 6), device="cuda")
    ids[prompt] = -1
    logits = torch.randn(300, 6, device="cuda")
    err, weights = B.new_err_word("cuda"), list(block.parameters())

    def step():
        loss = B.linear_distillation(block(*batch, err), block.vocab, ids, logits, 1.2, err_word=err)
        return [loss.detach(), *torch.autograd.grad(loss, weights)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(2):
        batch[0].mul_(-0.7)
        logits.add_(torch.randn_like(logits))
        ids[100 + k] = -1
        graph.replay()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_second_derivatives_are_refused():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    x = torch.randn(9, 64, device="cuda").bfloat16().requires_grad_()
    W = torch.randn(30, 64, device="cuda").bfloat16()
    q = torch.randn(9, 2, 64, device="cuda").bfloat16().requires_grad_()
    inv, _ = B.rope_frequencies(64)
    ids, t = torch.randint(0, 30, (9, 3), device="cuda"), torch.randn(9, 3, device="cuda")
    for leaf, out in ((x, B.linear_distillation(x, W, ids, t).pow(2)), (q, B.rope(q, q, inv)[0].float().pow(2).sum())):
        (g,) = torch.autograd.grad(out, leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.float().sum().backward()


def test_gradients_do_not_share_memory():
    """x and the residual get the same gradient, each in memory of its own."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    x, r = (torch.randn(9, 64, device="cuda").requires_grad_() for _ in range(2))
    y, s = B.layer_norm(x, None, residual=r)
    (y.pow(3).sum() + s.sum()).backward()
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    # one tensor on both sides, and rows that are one row in memory
    z = torch.randn(1, 64, device="cuda", requires_grad=True)
    wide = z.expand(9, 64)
    y, _ = B.layer_norm(wide, None, residual=wide)
    y.pow(3).sum().backward()
    v = z.detach().double().cpu().requires_grad_()
    torch.nn.functional.layer_norm(2 * v, (64,)).pow(3).sum().mul(9).backward()
    assert (z.grad.double().cpu() - v.grad).norm() <= 2e-5 * v.grad.norm()


@pytest.mark.parametrize("fp32", [False, True])
def test_gradients_and_inputs_off_their_alignment(fp32):
    """Autograd's own tensors may start anywhere: the entries copy what the kernels cannot
    read in place."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    dt = torch.float32 if fp32 else torch.bfloat16
    flat = torch.randn(10 * 128 + 4, device="cuda").to(dt)
    x = flat[3:3 + 1280].view(10, 128).requires_grad_()
    inv, _ = B.rope_frequencies(64)
    y = B.layer_norm(x, None, rms=True)
    a, b = B.rope(x.view(10, 2, 64), x.view(10, 2, 64), inv)
    torch.autograd.backward((y, a, b), (flat[1:1281].view(10, 128), flat[2:1282].view(10, 2, 64),
                                        flat[4:1284].view(10, 2, 64)))
    x2 = x.detach().clone().requires_grad_()
    y2 = B.layer_norm(x2, None, rms=True)
    a2, b2 = B.rope(x2.view(10, 2, 64), x2.view(10, 2, 64), inv)
    torch.autograd.backward((y2, a2, b2), (flat[1:1281].clone().view(10, 128), flat[2:1282].clone().view(10, 2, 64),
                                           flat[4:1284].clone().view(10, 2, 64)))
    assert torch.equal(y, y2) and torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(x.grad, x2.grad)
